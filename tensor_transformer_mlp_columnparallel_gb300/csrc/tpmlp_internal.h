// Host-side interfaces shared by the library's translation units (not part of
// the public C-ABI in include/tpmlp.h).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "tpmlp.h"

namespace tpmlp {

constexpr int kMaxG = TPMLP_MAX_SHARDS;

// What the GEMM epilogue does with each fp32 accumulator value v at (m, n):
//   EPI_STORE: C = v (+ bias[n])
//   EPI_ACT:   z = v (+ bias[n]); aux = z (if aux != NULL); C = act(z)
//   EPI_DACT:  C = v * act'(aux[m, n])
//   EPI_SWIGLU (dual GEMMs): g, u = the two accumulators at (m, n);
//              aux = g, aux2 = u (each if not NULL); C = SiLU(g) * u
//   EPI_DSWIGLU: g = aux[m, n], u = aux2[m, n], s = sigmoid(g);
//              C = v u s (1 + g (1 - s)) (dG), C2 = v g s (dU)
enum EpiKind { EPI_STORE = 0, EPI_ACT = 1, EPI_DACT = 2, EPI_SWIGLU = 3, EPI_DSWIGLU = 4 };

struct EpiArgs {
    int kind;
    int act;                   // tpmlp_act
    int out_f32;               // 1: C is fp32; 0: C has the compute element type
    int64_t ldc;               // row pitch of C, elements
    int64_t ldaux;             // row pitch of aux, elements
    void* C[kMaxG];            // per group (FOLD: group 0 only)
    const void* bias[kMaxG];   // per output column, compute element type; NULL: none
    void* aux[kMaxG];          // Z (compute element type), see EpiKind
    void* aux2[kMaxG];         // U of EPI_SWIGLU and EPI_DSWIGLU
    void* C2[kMaxG];           // dU of EPI_DSWIGLU, row pitch ldc
    // EPI_DSWIGLU, > 0: what rounding dG and dU to bf16 left over, itself in
    // bf16, this many bytes behind C and C2
    int64_t lo_off;
    // > 0: C is split by rows into blocks of row_shard rows, block i at C[i]
    // (the reduce-scatter output of the block end); 0: C[g] as above
    int64_t row_shard;
};

// A batch of G GEMMs of identical shape, C_g[M, N] = A_g[M, K] B_g[K, N], or,
// with fold = 1, ONE output C[M, N] = sum_g A_g B_g whose K loop runs over
// (g, k) in order g = 0..G-1.
// Operand addressing (elements):
//   A(m, k) = a_mn ? A[g][k * lda + m] : A[g][m * lda + k]
//   B(k, n) = b_mn ? B[g][k * ldb + n] : B[g][n * ldb + k]
// ("K-major" = the K index is contiguous; "MN-major" = M or N is contiguous.)
struct GemmProblem {
    int M, N, K;
    int G;
    int fold;
    const void* A[kMaxG];
    int64_t lda;
    int a_mn;
    const void* B[kMaxG];
    int64_t ldb;
    int b_mn;
    // dual = 1: a second B (B2, same layout as B) and two products per output,
    // A B and A B2, for the gated MLP's gate and up projections
    int dual;
    const void* B2[kMaxG];
    // chain = 1: the K loop of each group runs over two operand pairs, A B
    // and then A2 B2 (all K-major), into one accumulator: the
    // gated MLP's dX. With fold the order is (g, pair, k). Not with dual.
    int chain;
    const void* A2[kMaxG];
    // > 0 (chain, K-major A, M <= kRestRows): that many rows, M, behind A's (and
    // A2's) M hold what A's rounding left over, to be added to its products
    int rest_rows;
    EpiArgs epi;
    const char* name;          // kernel kind, for the timing records
    // Scratch for work-balanced few-token GEMMs (stream-K, M <= 64): partial
    // accumulator slots and per-tile arrival counters; NULL = not available.
    float* sk_part;
    size_t sk_part_bytes;
    int* sk_cnt;
    int64_t sk_cnt_cap;        // counters available
};

// Stream-K scratch: at most this many CTAs share the (tile, k-block) units,
// each with two slots of up to 64 rows x kSkMaxBn fp32 accumulators, and two
// counters per tile (one per 32-row warp).
constexpr int kSkMaxCtas = 256;
constexpr int kSkMaxBn = 256;

// bf16 inputs on tcgen05 tensor cores (TMA + mbarrier pipeline + TMEM).
tpmlp_status run_gemm_tc(const GemmProblem& p, cudaStream_t s);
// The tile configuration run_gemm_tc launches for p (accumulator columns,
// CTAs per MMA, K-split cluster size); nothing is launched.
tpmlp_status plan_gemm_tc(const GemmProblem& p, int* bn, int* mma_ctas, int* ksplit);
// fp32 inputs on CUDA cores (exact fp32 FMA, no TF32).
tpmlp_status run_gemm_simt(const GemmProblem& p, cudaStream_t s);

// bf16 weight gradients C[m, n] = sum_{k < K} A[k, m] (B + B2)[k, n] of few tokens
// k (M and N multiples of 8, pointers and pitches of 16 bytes; B2 NULL: none),
// all products of the list in one launch.
struct WeightGradProduct {
    const void* A;
    const void* B;
    const void* B2;
    void* C;
    int64_t lda, ldb, ldc;
    int M, N;
};
constexpr int kMaxWeightGrads = 3 * kMaxG;
constexpr int kRestRows = 16;   // both parts of a row among one warp's 32 accumulator rows
// Up to here the list's launch beats the grouped GEMMs (three products of 4096
// x 4096 by 4 shards on GB300: 61 us against 222 us at 16 tokens, 184 / 246 at
// 512, 311 / 280 at 1024): writing the outputs bounds it, not the MMAs.
constexpr int kFewTokens = 768;
tpmlp_status run_weight_grads(const WeightGradProduct* products, int count, int K, cudaStream_t s,
                              const char* name);

// Y = sum_r P[r] + bias, fp32 sum in shard order, output fp32 or bf16. With
// Y_rows != NULL the result is scattered by rows: rows [i*N/T, (i+1)*N/T) to
// Y_rows[i] (reduce-scatter); otherwise it goes to Y.
tpmlp_status run_block_reduce(int out_f32, int64_t N, int64_t D, int T, const float* const* P,
                              const void* bias, void* Y, cudaStream_t s, const char* name,
                              void* const* Y_rows = nullptr);
tpmlp_status run_vocab_embedding(int f32, int64_t N, int64_t V, int64_t H, int T,
                                 const int64_t* ids, const void* const* table, void* out,
                                 cudaStream_t s);
// out_g[c] = sum_r in_g[r * ld_g + c], c < cols_g, for G <= kMaxColsumG groups
// of `rows` rows each (bias gradients: the T dZ shards and dY). With fp32
// scratch space (scratch_bytes, 16-byte aligned; bf16 only) the sums stream
// whole rows in two passes through it, else one pass per column strip.
constexpr int kMaxColsumG = kMaxG + 1;
tpmlp_status run_colsum(int f32, int64_t rows, int G, const int64_t* cols, const int64_t* ld,
                        const void* const* in, void* const* out, cudaStream_t s,
                        float* scratch = nullptr, size_t scratch_bytes = 0);
tpmlp_status run_vocab_ce(int64_t N, int64_t V, int T, const float* logits,
                          const int64_t* targets, float* loss, float* loss_mean, int32_t* argmax,
                          int32_t* owner, cudaStream_t s);
tpmlp_status run_vocab_ce_backward(int64_t N, int64_t V, const float* logits,
                                   const int64_t* targets, const float* loss, float grad_scale,
                                   float* dlogits, cudaStream_t s);
// mean of loss[0..N), fixed order (NaN for N = 0)
tpmlp_status run_mean(const float* loss, int64_t N, float* out, cudaStream_t s);

// Token log probabilities, rank, entropy, lse and the K most likely tokens.
struct LogprobArgs {
    const void* logits;
    int64_t ld, N, V;
    int K;
    const int64_t* targets;    // NULL: no logprob, no rank
    float* logprob;
    int32_t* rank;
    float* entropy;
    float* lse;
    int32_t* top_ids;
    float* top_logprobs;
};
tpmlp_status run_vocab_logprobs(int f32, const LogprobArgs& a, cudaStream_t s);

// Distillation from a teacher's top tokens; what is NULL is not computed:
// loss (with lse) is the forward, dlogits the gradient. The gradient alone
// takes p from the forward's lse_in, where that is precise enough.
struct DistillArgs {
    const void* logits;
    int64_t ld, N, V;
    int K;
    const int32_t* ids;
    const float* teacher;
    float tau;
    float* loss;
    float* lse;
    const float* lse_in;
    const float* grad_tokens;
    float grad_scale;
    void* dlogits;
    int64_t ldd;
};
tpmlp_status run_vocab_distill(int f32, const DistillArgs& a, cudaStream_t s);

tpmlp_status run_vocab_embedding_scaled(int f32, int64_t N, int64_t V, int64_t H, int T,
                                        const int64_t* ids, const void* const* table, float scale,
                                        void* out, cudaStream_t s);
// Table gradient by sorted tokens (workspace laid out by embedding_grad_bytes).
size_t embedding_grad_bytes(int64_t N, int64_t V, int64_t H);
tpmlp_status run_vocab_embedding_backward(int f32, int grad_f32, int64_t N, int64_t V, int64_t H,
                                          int T, const int64_t* ids, const void* dout, float scale,
                                          int accumulate, void* const* dtable, void* workspace,
                                          cudaStream_t s);
tpmlp_status run_selftest_wait(uint64_t timeout_ns, cudaStream_t s);

// ---- services of the API translation unit --------------------------------
int* device_error_word();          // per current device; NULL on failure
uint64_t wait_timeout_ns();
int gemm_stall_role();             // failure-detection self test of the GEMM (0: off)
int weight_grad_stall_role();      // of the few-token weight gradients: their own, else the GEMM's
bool pdl_enabled();                // programmatic dependent launch (TPMLP_PDL != 0)
bool alternate_orders();           // odd waves walk K down, odd bands their tiles back (TPMLP_ALT_ORDER != 0)
int device_sm_count();

// Counts the launch and, when timing is on, brackets it with CUDA events
// recorded on the launch stream.
class LaunchScope {
  public:
    LaunchScope(const char* name, cudaStream_t s);
    ~LaunchScope();

  private:
    const char* name_;
    cudaStream_t s_;
    cudaEvent_t start_;
    cudaEvent_t stop_;
};

}  // namespace tpmlp
