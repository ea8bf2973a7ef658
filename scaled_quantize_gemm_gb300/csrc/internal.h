// internal.h -- host-side launcher interface between the C-ABI layer
// (api.cu) and the kernel translation units.  Not installed, not part of the ABI.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fp8sq {

enum { kE4M3 = 0, kE5M2 = 1 };
enum { kBF16 = 0, kF32 = 1 };
enum { kTensor = 0, kTile = 1, kBlock = 2, kMX = 3, kMXTiled = 4, kTileCol = 5, kMXCol = 6,
       kTilePow2 = 7, kBlockPow2 = 8, kMXFloor = 9,
       kTileRowCol = 10, kMXRowCol = 11,     // rows and columns in one pass (fp8_quantize_rows_cols)
       kTileRowColPow2 = 12 };               // the same for power-of-two 1x128 / 128x1 tiles, tiled E8M0 codes

struct QuantArgs {
    const void* x = nullptr;
    int x_dtype = kBF16;
    int64_t rows = 0, cols = 0;
    int format = kE4M3;
    int gran = kTensor;
    float* state = nullptr;          // delayed state block (TENSOR only) or null
    int history_len = 0;
    uint8_t* q = nullptr;            // may be null only for amax-only launches
    uint8_t* qT = nullptr;
    void* scales = nullptr;
    float* scalesT = nullptr;        // 128x128 blocks with qT: the transposed scale grid (power-of-two
                                     // blocks: the tiled E8M0 codes of x^T, as bytes)
    void* col_scales = nullptr;      // rows and columns in one pass: the column-unit scales
    float* amax = nullptr;
    unsigned long long* sat = nullptr;
    const float* amax_in = nullptr;  // current per-tensor: the amax of pass 1
};

// quantize.cu
cudaError_t launch_amax(const QuantArgs& a, cudaStream_t st, int sms);    // writes a.amax per unit
cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t st, int sms);
// two per-tensor casts with transposed copies (same dtype, format and
// recipe) in one launch; other argument pairs go through launch_quantize twice
cudaError_t launch_quantize_pair(const QuantArgs& a, const QuantArgs& b, cudaStream_t st, int sms);
cudaError_t launch_scale_init(float* states, int n, int H, cudaStream_t st);
cudaError_t launch_update_scale(float* states, int n, int H, const int* formats, int algo, cudaStream_t st);
// LayerNorm of bf16 x [rows][cols] fused into the delayed per-tensor cast
// (a.state required); writes mu, rstd [rows]
cudaError_t launch_layernorm_quantize(const QuantArgs& a, const float* gamma, const float* beta, float eps,
                                      float* mu, float* rstd, cudaStream_t st, int sms);

struct GemmArgs {
    const uint8_t* A = nullptr;
    const uint8_t* B = nullptr;
    int a_format = kE4M3, b_format = kE4M3;
    int mode = 0;                    // 0 per-tensor, 1 tile x block promotion, 2 MX (tiled E8M0 scales),
                                     // 3 column tiles x column tiles (promotion, scales [K/128][rows])
    const void* a_scale = nullptr;
    const void* b_scale = nullptr;
    int64_t M = 0, N = 0, K = 0;
    const float* bias = nullptr;
    void* D = nullptr;
    int d_dtype = kBF16;
    // operand storage (mode 0 only): K-major A [M][K] / B [N][K], or
    // MN-major A [K][M] / B [K][N]
    bool a_mn = false, b_mn = false;
    // mode 0, bf16 D only: also cast D to FP8 codes q_out [M][N] with the
    // delayed per-tensor state q_state (history q_history_len)
    uint8_t* q_out = nullptr;
    float* q_state = nullptr;
    int q_history_len = 0, q_format = kE4M3;
};

// gemm.cu
cudaError_t launch_gemm(const GemmArgs& g, cudaStream_t st, int sms, const char** why);
// Raises a kernel's dynamic shared-memory limit to `bytes`, once per device.
cudaError_t smem_attr_once(const void* kern, int bytes);
// device address of the GEMM kernels' error word on the current device
cudaError_t device_error_word(int** word);
int gemm_ctas(const GemmArgs& g, int sms);   // SMs its persistent grid occupies, -1 if unknown
int read_device_error(int clear);   // 0 or the GEMM kernels' device error word
// launches a kernel whose bounded wait is made to run out (failure-path test)
cudaError_t launch_selftest_wait(uint64_t limit_ns, int* waited_out, cudaStream_t st);
// 2-D tiled TMA map, 128-byte swizzle, zero fill out of bounds; u16 selects
// 2-byte elements (else 1-byte)
bool encode_tmap_2d(CUtensorMap* m, int u16, const void* ptr, uint64_t inner, uint64_t rows, uint32_t box_inner,
                    uint32_t box_rows);

// ffn.cu: products with their elementwise work in the epilogue (per-tensor scales)
enum { kFfnAct = 0, kFfnGlu = 1, kFfnGluBwd = 2 };
struct FfnArgs {
    int kind = kFfnAct;
    int64_t M = 0, N = 0, K = 0;     // N: output columns (glu: features F, B is [2F][K]; glu_bwd: B is [K][F])
    const uint8_t* A = nullptr;
    const uint8_t* B = nullptr;
    int a_format = kE4M3, b_format = kE4M3;
    const float* a_scale = nullptr;
    const float* b_scale = nullptr;
    int act = 0;
    const float* bias = nullptr;
    const void* residual = nullptr;
    int res_dtype = kBF16;
    void* D = nullptr;
    int d_dtype = kBF16;
    void* Z = nullptr;               // bf16 [M][N] (glu: [M][2F])
    const void* gu = nullptr;        // glu_bwd: bf16 [M][2F]
    uint8_t* q_out = nullptr;        // [M][N] (glu_bwd: [M][2F])
    int q_format = kE4M3;
    float* q_state = nullptr;
    int q_history_len = 0;
    void* workspace = nullptr;       // ffn_workspace bytes, or null
};
size_t ffn_workspace(int kind, int64_t M, int64_t N, int64_t K);
cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t st, int sms, const char** why);

// rowops.cu: LayerNorm forward / backward, the elementwise backward of an
// activation with its bias gradient
struct LnArgs {
    int64_t M = 0, K = 0;
    int dtype = kBF16;               // of x, residual, sum, y, dy, dres, dx
    const void* x = nullptr;
    const float* gamma = nullptr;
    const float* beta = nullptr;
    float eps = 0.0f;
    const void* residual = nullptr;  // forward: added to x
    void* sum = nullptr;             // forward: x + residual as rounded
    void* y = nullptr;
    uint8_t* q = nullptr;            // forward: codes of y under a delayed state, or null
    int q_format = kE4M3;
    float* q_state = nullptr;
    int q_history_len = 0;
    int q_gran = kTensor;            // RMSNorm: the codes' scaling unit (kTensor: the delayed state)
    void* q_scales = nullptr;
    float* mu = nullptr;
    float* rstd = nullptr;
    const void* dy = nullptr;        // backward
    const void* dres = nullptr;
    void* dx = nullptr;
    float* dgamma = nullptr;
    float* dbeta = nullptr;
    void* workspace = nullptr;
};
cudaError_t launch_layernorm_fwd(const LnArgs& a, cudaStream_t st, int sms);
cudaError_t launch_layernorm_bwd(const LnArgs& a, cudaStream_t st, int sms);
size_t layernorm_bwd_workspace(int64_t M, int64_t K);
// rmsnorm.cu (mu, beta and dbeta unused)
cudaError_t launch_rmsnorm_fwd(const LnArgs& a, cudaStream_t st, int sms);
cudaError_t launch_rmsnorm_bwd(const LnArgs& a, cudaStream_t st, int sms);
size_t rmsnorm_bwd_workspace(int64_t M, int64_t K);
struct ActBwdArgs {
    int64_t M = 0, N = 0;
    const void* dy = nullptr;        // bf16
    const void* z = nullptr;         // bf16
    int act = 0;
    float* dbias = nullptr;
    void* dz = nullptr;              // bf16 or null
    uint8_t* q = nullptr;
    int q_format = kE5M2;
    float* q_state = nullptr;
    int q_history_len = 0;
    void* workspace = nullptr;
};
cudaError_t launch_act_bwd(const ActBwdArgs& a, cudaStream_t st, int sms);
size_t act_bwd_workspace(int64_t M, int64_t N);

// experts_rows.cu: rows sorted by expert and back
constexpr int kExpertPad = 32;       // an expert's segment of the sorted rows is a multiple of this
constexpr int kExpertTile = 256;     // rows of a product's tile
constexpr int kExpertGroup = 8;      // neighbouring tiles of one expert that share the weights' tiles in L2
constexpr int kExpertMax = 1024;     // experts
constexpr int kExpertSlots = 64;     // experts of a token
// The plan of a routing, int32: offsets [E + 1], counts [E], the number of row
// tiles; at tiles_at the tiles, four each {first tile of its group, expert << 8
// | tiles in the group, the group's first row, the expert's last row + 1}; at
// blocks_at every block of 32 rows, four each {expert, the expert's first block,
// its blocks, rows of the block that are not padding}; at row_of_at the sorted
// row of every assignment, or -1.
struct ExpertLayout {
    int64_t rows = 0, max_tiles = 0, tiles_at = 0, blocks_at = 0, row_of_at = 0, ints = 0;
};
ExpertLayout expert_layout(int64_t T, int k, int E);
struct ExpertRowsArgs {
    int64_t T = 0, K = 0;
    int k = 0, E = 0;
    ExpertLayout layout;
    const int32_t* ids = nullptr;
    int32_t* plan_out = nullptr;
    const int32_t* plan = nullptr;
    const void* x = nullptr;         // dispatch: [T][K] of `size` bytes an element
    int size = 1;
    void* rows_out = nullptr;
    int dtype = kBF16;               // combine and its backward pass
    const void* rows = nullptr;
    const float* weights = nullptr;
    const void* residual = nullptr;
    void* y = nullptr;
    const void* dy = nullptr;
    void* drows = nullptr;
    float* dweights = nullptr;
    uint8_t* q = nullptr;
    int q_format = kE5M2;
    float* q_state = nullptr;
    int q_history_len = 0;
};
cudaError_t launch_expert_plan(const ExpertRowsArgs& a, cudaStream_t st);
cudaError_t launch_expert_dispatch(const ExpertRowsArgs& a, cudaStream_t st, int sms);
cudaError_t launch_expert_combine(const ExpertRowsArgs& a, cudaStream_t st, int sms);
cudaError_t launch_expert_combine_bwd(const ExpertRowsArgs& a, cudaStream_t st, int sms);

// experts.cu: the experts' products (per-tensor scale of A, a scale for each
// expert's B)
enum { kExpertGemm = 0, kExpertGlu = 1, kExpertGluBwd = 2, kExpertWgrad = 3 };
struct ExpertGemmArgs {
    int kind = kExpertGemm;
    int64_t T = 0;
    int k = 0, E = 0;
    ExpertLayout layout;
    const int32_t* plan = nullptr;
    int64_t M = 0, N = 0, K = 0;     // M: wgrad (rows of each D); N: columns (glu: features); K: contraction
    bool b_mn = false;               // gemm: B [E][K][N]
    const uint8_t* A = nullptr;
    const uint8_t* B = nullptr;
    int a_format = kE4M3, b_format = kE4M3;
    const float* a_scale = nullptr;
    const float* b_scale = nullptr;  // [E] (wgrad: one)
    int act = 0;
    const void* gu = nullptr;        // glu_bwd: bf16 [R][2F]
    void* D = nullptr;               // gemm [R][N], glu h bf16 [R][F], wgrad [E][M][N]
    int d_dtype = kBF16;
    void* Z = nullptr;               // glu: bf16 [R][2F]
    uint8_t* q_out = nullptr;
    int q_format = kE4M3;
    float* q_state = nullptr;
    int q_history_len = 0;
    void* workspace = nullptr;
};
cudaError_t launch_expert_gemm(const ExpertGemmArgs& a, cudaStream_t st, int sms, const char** why);
size_t expert_workspace(int64_t T, int k, int E, int64_t N, int64_t K);

// api.cu: the calling thread's error message and the sm_103 device check
int api_fail(int code, const char* fmt, ...);
int api_check_device(int* sms);

}  // namespace fp8sq
