// Kernel-level C ABI (gpt2_kernels.h): single operations on caller-owned
// device buffers.
#include <string>

#include "gpt2_kernels.h"
#include "kernels.cuh"

using namespace gpt2;

namespace gpt2 {
int set_error(int code, const char* msg);   // defined in gpt2_api.cu
}

extern "C" int gpt2k_matmul_bf16(int layout, const void* A, const void* B, int M, int N, int K, int epilogue,
                                 void* out, int64_t ldo, void* out2, const float* bias, const float* resid,
                                 const void* aux, float* colsum_part, float beta, int engine,
                                 uint32_t* status_dev, void* stream) {
    if (layout < GPT2K_NT || layout > GPT2K_TN) return set_error(GPT2_ERR_INVALID_ARG, "unknown layout");
    if (epilogue < GPT2K_EPI_STORE || epilogue > GPT2K_EPI_ACCUM_F32)
        return set_error(GPT2_ERR_INVALID_ARG, "unknown epilogue");
    if (M < 1 || N < 1 || K < 1 || ldo < N) return set_error(GPT2_ERR_INVALID_ARG, "bad sizes");
    if (!A || !B || !out || !status_dev) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    const bool needs_bias = epilogue == GPT2K_EPI_BIAS || epilogue == GPT2K_EPI_BIAS_GELU ||
                            epilogue == GPT2K_EPI_BIAS_RESID;
    if ((needs_bias && !bias) || (epilogue == GPT2K_EPI_BIAS_GELU && !out2) ||
        (epilogue == GPT2K_EPI_BIAS_RESID && !resid) || (epilogue == GPT2K_EPI_MUL && !aux))
        return set_error(GPT2_ERR_INVALID_ARG, "epilogue operand missing");
    if (colsum_part && (epilogue != GPT2K_EPI_MUL || engine != 1))
        return set_error(GPT2_ERR_INVALID_ARG, "column sums come only with the tensor-core GPT2K_EPI_MUL epilogue");
    long long launches = 0;
    Ctx c;
    c.stream = (cudaStream_t)stream;
    c.status = status_dev;
    c.launches = &launches;
    c.num_sms = 148;
    Epilogue e;
    e.kind = epilogue;
    e.out = out;
    e.ldo = ldo;
    e.out2 = out2;
    e.bias = bias;
    e.resid = resid;
    e.aux = aux;
    e.colsum_part = colsum_part;
    e.beta = beta;
    const GemmLayout L = (GemmLayout)layout;
    if (engine == 1) {
        if (!gemm_tc_supported(L, M, N, K))
            return set_error(GPT2_ERR_INVALID_ARG, "shape not supported by the tensor-core GEMM");
        if (ldo % 8 != 0) return set_error(GPT2_ERR_INVALID_ARG, "the tensor-core GEMM needs ldo % 8 == 0");
        if (epilogue == GPT2K_EPI_ACCUM_F32 && beta != 0.f && beta != 1.f)
            return set_error(GPT2_ERR_INVALID_ARG, "the tensor-core GEMM accumulates with beta 0 or 1");
        if (!launch_gemm_tc(c, L, (const bf16*)A, (const bf16*)B, M, N, K, e))
            return set_error(GPT2_ERR_CUDA, "tensor-map encoding failed");
    } else {
        launch_gemm_simt<bf16>(c, L, (const bf16*)A, (const bf16*)B, M, N, K, e);
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

namespace {
int check_attention_args(int dtype, int B, int T, int H, int hd, int engine, const void* a, const void* b,
                         const void* c, const uint32_t* status) {
    if (dtype != GPT2K_F32 && dtype != GPT2K_BF16) return set_error(GPT2_ERR_INVALID_ARG, "unknown dtype");
    if (B < 1 || T < 1 || H < 1) return set_error(GPT2_ERR_INVALID_ARG, "B, T, H must be >= 1");
    if (hd != 32 && hd != 64) return set_error(GPT2_ERR_INVALID_ARG, "head width must be 32 or 64");
    if (engine < 0 || engine > 2) return set_error(GPT2_ERR_INVALID_ARG, "unknown attention engine");
    if (engine >= 1 && dtype != GPT2K_BF16)
        return set_error(GPT2_ERR_INVALID_ARG, "the tensor-core attention engines take bf16 operands");
    if (engine == 2 && hd != 64)
        return set_error(GPT2_ERR_INVALID_ARG, "the tcgen05 attention engine needs head width 64");
    if (!a || !b || !c || !status) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    return GPT2_OK;
}

Ctx kctx(void* stream, uint32_t* status, long long* launches) {
    Ctx c;
    c.stream = (cudaStream_t)stream;
    c.status = status;
    c.launches = launches;
    c.num_sms = 148;
    return c;
}
}  // namespace

extern "C" int gpt2k_attention_fwd(int dtype, const void* qkv, void* out, float* lse, int B, int T, int H, int hd,
                                   int engine, uint32_t* status_dev, void* stream) {
    int rc = check_attention_args(dtype, B, T, H, hd, engine, qkv, out, lse, status_dev);
    if (rc) return rc;
    long long launches = 0;
    Ctx c = kctx(stream, status_dev, &launches);
    if (engine == 2) {
        if (!launch_attention_fwd_tc(c, (const bf16*)qkv, (bf16*)out, lse, B, T, H))
            return set_error(GPT2_ERR_CUDA, "tensor-map encoding failed");
    } else if (engine == 1)
        launch_attention_fwd_mma(c, (const bf16*)qkv, (bf16*)out, lse, B, T, H, hd);
    else if (dtype == GPT2K_F32)
        launch_attention_fwd_simt<float>(c, (const float*)qkv, (float*)out, lse, B, T, H, hd);
    else
        launch_attention_fwd_simt<bf16>(c, (const bf16*)qkv, (bf16*)out, lse, B, T, H, hd);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

namespace {
// engine 2 workspace: [D: B*H*T floats, padded to 64][dQ accumulator: B*T*C floats][work counter: 64]
long long attention_bwd_dq_offset(int B, int T, int H) { return ((long long)B * H * T + 63) / 64 * 64; }
long long attention_bwd_work_offset(int B, int T, int H, int hd) {
    return attention_bwd_dq_offset(B, T, H) + ((long long)B * T * H * hd + 63) / 64 * 64;
}
}  // namespace

extern "C" int gpt2k_attention_bwd_workspace(int B, int T, int H, int hd, int engine, int64_t* floats) {
    if (!floats) return set_error(GPT2_ERR_INVALID_ARG, "NULL argument");
    if (B < 1 || T < 1 || H < 1 || (hd != 32 && hd != 64) || engine < 0 || engine > 2)
        return set_error(GPT2_ERR_INVALID_ARG, "bad size, head width or engine");
    *floats = engine == 2 ? attention_bwd_work_offset(B, T, H, hd) + 64 : (long long)B * H * T;
    return GPT2_OK;
}

extern "C" int gpt2k_attention_bwd(int dtype, const void* qkv, const void* out, const void* dout, const float* lse,
                                   void* dqkv, int B, int T, int H, int hd, float* workspace_dev,
                                   float* colsum_part, int engine, uint32_t* status_dev, void* stream) {
    int rc = check_attention_args(dtype, B, T, H, hd, engine, qkv, out, dout, status_dev);
    if (rc) return rc;
    if (!lse || !dqkv || !workspace_dev) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    if (colsum_part && engine != 2)
        return set_error(GPT2_ERR_INVALID_ARG, "column sums come only with the tcgen05 attention backward");
    long long launches = 0;
    Ctx c = kctx(stream, status_dev, &launches);
    if (engine == 2) {
        if (!launch_attention_bwd_tc(c, (const bf16*)qkv, (const bf16*)out, (const bf16*)dout, lse, workspace_dev,
                                     workspace_dev + attention_bwd_dq_offset(B, T, H),
                                     (int*)(workspace_dev + attention_bwd_work_offset(B, T, H, hd)), (bf16*)dqkv, B,
                                     T, H, colsum_part))
            return set_error(GPT2_ERR_CUDA, "tensor-map encoding failed");
    } else if (engine == 1)
        launch_attention_bwd_mma(c, (const bf16*)qkv, (const bf16*)out, (const bf16*)dout, lse, workspace_dev,
                                 (bf16*)dqkv, B, T, H, hd);
    else if (dtype == GPT2K_F32)
        launch_attention_bwd_simt<float>(c, (const float*)qkv, (const float*)out, (const float*)dout, lse,
                                         workspace_dev, (float*)dqkv, B, T, H, hd);
    else
        launch_attention_bwd_simt<bf16>(c, (const bf16*)qkv, (const bf16*)out, (const bf16*)dout, lse,
                                        workspace_dev, (bf16*)dqkv, B, T, H, hd);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

extern "C" int gpt2k_attention_decode(int dtype, const void* cache, void* out, int B, int H, int hd, int Tc, int n,
                                      float* workspace_dev, uint32_t* status_dev, void* stream) {
    if (dtype != GPT2K_F32 && dtype != GPT2K_BF16) return set_error(GPT2_ERR_INVALID_ARG, "unknown dtype");
    if (B < 1 || H < 1 || Tc < 1 || n < 1 || n > Tc)
        return set_error(GPT2_ERR_INVALID_ARG, "need B, H >= 1 and 1 <= n <= Tc");
    if (hd != 32 && hd != 64) return set_error(GPT2_ERR_INVALID_ARG, "head width must be 32 or 64");
    if ((H * hd) % 64 != 0) return set_error(GPT2_ERR_INVALID_ARG, "C = H * hd must be a multiple of 64");
    if (!cache || !out || !workspace_dev || !status_dev) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    long long launches = 0;
    Ctx c = kctx(stream, status_dev, &launches);
    if (dtype == GPT2K_F32)
        launch_attention_decode<float>(c, (const float*)cache, (float*)out, workspace_dev, B, H, hd, Tc, n);
    else
        launch_attention_decode<bf16>(c, (const bf16*)cache, (bf16*)out, workspace_dev, B, H, hd, Tc, n);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

extern "C" int gpt2k_sample(int dtype, const void* logits, int rows, int V, int64_t ld, float temperature,
                            int top_k, const float* u_dev, int32_t* next_dev, uint32_t* status_dev, void* stream) {
    if (dtype != GPT2K_F32 && dtype != GPT2K_BF16) return set_error(GPT2_ERR_INVALID_ARG, "unknown dtype");
    if (rows < 1 || V < 1 || ld < V) return set_error(GPT2_ERR_INVALID_ARG, "need rows, V >= 1 and ld >= V");
    if (!logits || !u_dev || !next_dev || !status_dev) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    if (!(temperature > 0.f) || !(temperature < INFINITY))
        return set_error(GPT2_ERR_INVALID_ARG, "temperature must be finite and > 0");
    long long launches = 0;
    Ctx c = kctx(stream, status_dev, &launches);
    if (dtype == GPT2K_F32)
        launch_sample<float>(c, (const float*)logits, ld, rows, V, temperature, top_k, u_dev, next_dev, nullptr, 0, 0);
    else
        launch_sample<bf16>(c, (const bf16*)logits, ld, rows, V, temperature, top_k, u_dev, next_dev, nullptr, 0, 0);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

extern "C" int gpt2k_embedding_bwd_workspace(int B, int T, int C, int64_t* floats) {
    if (B < 1 || T < 1 || C < 1 || !floats) return set_error(GPT2_ERR_INVALID_ARG, "need B, T, C >= 1 and floats");
    *floats = (int64_t)embed_bwd_scratch_floats((long long)B * T, C);
    return GPT2_OK;
}

extern "C" int gpt2k_embedding_bwd(const int32_t* idx, const float* dx, int B, int T, int C, int V, float* dwte,
                                   float* dwpe, float* workspace_dev, uint32_t* status_dev, void* stream) {
    if (B < 1 || T < 1 || C < 1 || V < 1) return set_error(GPT2_ERR_INVALID_ARG, "need B, T, C, V >= 1");
    if (C % 4 != 0) return set_error(GPT2_ERR_INVALID_ARG, "C must be a multiple of 4");
    if (!idx || !dx || !dwte || !dwpe || !status_dev) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    long long launches = 0;
    Ctx c = kctx(stream, status_dev, &launches);
    launch_embed_bwd(c, idx, dx, B, T, C, V, dwte, dwpe, workspace_dev);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

// ---------------------------------------------------------------- 8-bit linear layers
namespace {
bool misaligned(const void* p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }
size_t elem_size(int dtype) { return dtype == GPT2K_F32 ? 4 : 2; }
// Programmatic dependent launch: the call's blocks start while the kernel before it in the stream ends,
// and wait for it (griddep_wait) before they touch memory. About 1 us less between small calls.
Ctx early_kctx(void* stream, uint32_t* status, long long* launches) {
    Ctx c = kctx(stream, status, launches);
    c.pdl = true;
    return c;
}
constexpr int MAX_EXTENT = 1 << 30;   // rows, columns: 32-bit index arithmetic has room past them
}  // namespace

extern "C" int gpt2k_quantize_rows(int dtype, const void* x, int rows, int K, int64_t ldx, int8_t* q, int64_t ldq,
                                   float* scale, void* stream) {
    if (dtype != GPT2K_F32 && dtype != GPT2K_BF16) return set_error(GPT2_ERR_INVALID_ARG, "unknown dtype");
    if (rows < 1 || K < 1 || ldx < K || ldq < K)
        return set_error(GPT2_ERR_INVALID_ARG, "need rows, K >= 1 and row strides >= K");
    if (rows > MAX_EXTENT || K > MAX_EXTENT) return set_error(GPT2_ERR_INVALID_ARG, "rows or K above 2^30");
    if (!x || !q || !scale) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    if (misaligned(x, elem_size(dtype)) || misaligned(scale, 4))
        return set_error(GPT2_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    long long launches = 0;
    Ctx c = early_kctx(stream, nullptr, &launches);
    if (dtype == GPT2K_F32)
        launch_quantize_rows<float>(c, (const float*)x, ldx, rows, K, q, ldq, scale);
    else
        launch_quantize_rows<bf16>(c, (const bf16*)x, ldx, rows, K, q, ldq, scale);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

extern "C" int gpt2k_matmul_i8(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                               const float* b_scale, int M, int N, int K, int epilogue, int out_dtype, void* out,
                               int64_t ldo, const float* bias, const float* resid, int64_t ldr, uint32_t* status_dev,
                               void* stream) {
    if (epilogue < GPT2K_EPI_STORE || epilogue > GPT2K_EPI_BIAS_RESID)
        return set_error(GPT2_ERR_INVALID_ARG, "the int8 product has the epilogues store, bias, bias_gelu, bias_resid");
    if (out_dtype != GPT2K_F32 && out_dtype != GPT2K_BF16) return set_error(GPT2_ERR_INVALID_ARG, "unknown dtype");
    if (M < 1 || N < 1 || K < 1 || lda < K || ldb < K || ldo < N)
        return set_error(GPT2_ERR_INVALID_ARG, "need M, N, K >= 1, lda, ldb >= K and ldo >= N");
    if (M > MAX_EXTENT || N > MAX_EXTENT) return set_error(GPT2_ERR_INVALID_ARG, "M or N above 2^30");
    if (K > I8_MAX_K) return set_error(GPT2_ERR_INVALID_ARG, "K above 131071: a 32-bit sum could overflow");
    if (!A || !a_scale || !B || !b_scale || !out || !status_dev) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    if (epilogue != GPT2K_EPI_STORE && !bias) return set_error(GPT2_ERR_INVALID_ARG, "epilogue operand missing");
    if (epilogue == GPT2K_EPI_BIAS_RESID) {
        if (!resid) return set_error(GPT2_ERR_INVALID_ARG, "epilogue operand missing");
        if (out_dtype != GPT2K_F32) return set_error(GPT2_ERR_INVALID_ARG, "bias_resid writes fp32");
        if (ldr < N) return set_error(GPT2_ERR_INVALID_ARG, "need ldr >= N");
        if (resid == out && ldr != ldo && M > 1)
            return set_error(GPT2_ERR_INVALID_ARG, "a result in place of the residual has its row stride");
    }
    if (misaligned(a_scale, 4) || misaligned(b_scale, 4) || misaligned(out, elem_size(out_dtype)) ||
        misaligned(bias, 4) || misaligned(resid, 4) || misaligned(status_dev, 4))
        return set_error(GPT2_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    long long launches = 0;
    Ctx c = early_kctx(stream, status_dev, &launches);
    I8Product p;
    p.A = A;
    p.lda = lda;
    p.sa = a_scale;
    p.B = B;
    p.ldb = ldb;
    p.sb = b_scale;
    p.M = M;
    p.N = N;
    p.K = K;
    p.kind = epilogue;
    p.out_f32 = out_dtype == GPT2K_F32;
    p.out = out;
    p.ldo = ldo;
    p.bias = bias;
    p.resid = resid;
    p.ldr = ldr;
    if (!launch_matmul_i8(c, p)) {
        cudaError_t err = cudaGetLastError();   // read, so that no later call reports it
        return set_error(GPT2_ERR_CUDA, err != cudaSuccess ? cudaGetErrorString(err) : "tensor-map encoding failed");
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

// ---------------------------------------------------------------- token log-probabilities
namespace {
int check_logprob_args(int dtype, const void* logits, int rows, int V, int64_t ld, float temperature,
                       const uint32_t* status) {
    if (dtype != GPT2K_F32 && dtype != GPT2K_BF16) return set_error(GPT2_ERR_INVALID_ARG, "unknown dtype");
    if (rows < 1 || V < 1 || ld < V) return set_error(GPT2_ERR_INVALID_ARG, "need rows, V >= 1 and ld >= V");
    if (!logits || !status) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    if (!(temperature > 0.f) || !(temperature <= LOGPROB_MAX_TEMPERATURE) || !(1.5f / temperature < INFINITY))
        return set_error(GPT2_ERR_INVALID_ARG, "temperature must be > 0 and at most 1e20, 1.5 / temperature finite");
    if (V > MAX_EXTENT || (long long)rows * (V / 2048 + 1) > MAX_EXTENT)
        return set_error(GPT2_ERR_INVALID_ARG, "V above 2^30, or rows x V more than one launch takes");
    if (misaligned(logits, elem_size(dtype)) || misaligned(status, 4))
        return set_error(GPT2_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    return GPT2_OK;
}
}  // namespace

extern "C" int gpt2k_token_logprobs(int dtype, const void* logits, int rows, int V, int64_t ld, float temperature,
                                    const int32_t* targets, int top_k, float* logp, float* entropy, float* lse,
                                    int32_t* top_ids, float* top_logp, uint32_t* status_dev, void* stream) {
    int rc = check_logprob_args(dtype, logits, rows, V, ld, temperature, status_dev);
    if (rc) return rc;
    if ((targets != nullptr) != (logp != nullptr))
        return set_error(GPT2_ERR_INVALID_ARG, "targets and logp are given together");
    if (top_k < 0 || top_k > LOGPROB_MAX_TOP || top_k > V)
        return set_error(GPT2_ERR_INVALID_ARG, "need 0 <= top_k <= min(32, V)");
    if ((top_k > 0) != (top_ids != nullptr) || (top_k > 0) != (top_logp != nullptr))
        return set_error(GPT2_ERR_INVALID_ARG, "top_ids and top_logp are given exactly when top_k > 0");
    if (!logp && !entropy && !lse && !top_k) return set_error(GPT2_ERR_INVALID_ARG, "no output asked for");
    if (misaligned(targets, 4) || misaligned(logp, 4) || misaligned(entropy, 4) || misaligned(lse, 4) ||
        misaligned(top_ids, 4) || misaligned(top_logp, 4))
        return set_error(GPT2_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    long long launches = 0;
    Ctx c = early_kctx(stream, status_dev, &launches);
    const LogprobOut o = {logp, entropy, lse, top_ids, top_logp, top_k};
    if (dtype == GPT2K_F32)
        launch_token_logprobs<float>(c, (const float*)logits, ld, rows, V, temperature, targets, o);
    else
        launch_token_logprobs<bf16>(c, (const bf16*)logits, ld, rows, V, temperature, targets, o);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}

extern "C" int gpt2k_token_logprobs_bwd(int dtype, const void* logits, int rows, int V, int64_t ld, float temperature,
                                        const int32_t* targets, const float* lse, const float* dlogp,
                                        const float* entropy, const float* dentropy, void* dlogits, int64_t ldd,
                                        uint32_t* status_dev, void* stream) {
    int rc = check_logprob_args(dtype, logits, rows, V, ld, temperature, status_dev);
    if (rc) return rc;
    if (ldd < V) return set_error(GPT2_ERR_INVALID_ARG, "need ldd >= V");
    if (!lse || !dlogits) return set_error(GPT2_ERR_INVALID_ARG, "NULL operand");
    if (!dlogp && !dentropy) return set_error(GPT2_ERR_INVALID_ARG, "need dlogp or dentropy");
    if ((dlogp != nullptr) != (targets != nullptr))
        return set_error(GPT2_ERR_INVALID_ARG, "targets and dlogp are given together");
    if (dentropy && !entropy) return set_error(GPT2_ERR_INVALID_ARG, "dentropy needs entropy");
    if (dlogits == logits && ldd != ld)
        return set_error(GPT2_ERR_INVALID_ARG, "a gradient in place of the logits has their row stride");
    if (misaligned(dlogits, elem_size(dtype)) || misaligned(targets, 4) || misaligned(lse, 4) ||
        misaligned(dlogp, 4) || misaligned(entropy, 4) || misaligned(dentropy, 4))
        return set_error(GPT2_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
    long long launches = 0;
    Ctx c = early_kctx(stream, status_dev, &launches);
    if (dtype == GPT2K_F32)
        launch_token_logprobs_bwd<float>(c, (const float*)logits, ld, rows, V, temperature, targets, lse, dlogp,
                                         entropy, dentropy, (float*)dlogits, ldd);
    else
        launch_token_logprobs_bwd<bf16>(c, (const bf16*)logits, ld, rows, V, temperature, targets, lse, dlogp, entropy,
                                        dentropy, (bf16*)dlogits, ldd);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(GPT2_ERR_CUDA, cudaGetErrorString(err));
    return GPT2_OK;
}
