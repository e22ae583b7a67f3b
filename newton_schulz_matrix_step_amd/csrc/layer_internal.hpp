// Arguments and launch wrappers of the layer operators (layer_api.cpp on the
// host, norm_kernels.hip and linear_kernels.hip on the device), and the part of
// a handle that both API sources use.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <memory>
#include <string>

struct muon_handle;

namespace muon {

// State the layer operators keep on a handle (their workspaces).  Freed by
// muon_destroy after the device is idle, with the handle's device current.
struct HandleExt {
    virtual ~HandleExt() = default;
    virtual int64_t workspace_bytes() const = 0;
};

struct HandleBase {
    int device = 0;
    uint32_t flags = 0;
    std::string err;
    std::unique_ptr<HandleExt> layers;
};

HandleBase* handle_base(muon_handle* h);   // muon_api.cpp

constexpr int kAct8Group = 32;             // columns that share one exponent

// A launch has fewer than 2^32 threads along a dimension of its grid.  Passes
// over the rows of one matrix go in slices of at most 2^31 (MUON_SLICE_THREADS:
// smaller in a build that checks them); a product or a norm of long rows that
// would need more is refused.
#ifndef MUON_SLICE_THREADS
#define MUON_SLICE_THREADS (int64_t(1) << 31)
#endif
constexpr int64_t kGridThreads = int64_t(1) << 32;
constexpr int64_t kSliceThreads = MUON_SLICE_THREADS;
constexpr int64_t kMaxTiles128 = kGridThreads / 256 - 8;   // 128-wide output tiles, of 256 threads, in eighths

// 8-bit checkpoint as the kernels take it: element (r, c) is
// codes[r * ld + c] * 2^(exps[r * lde + c / 32] - 127).
struct Act8View {
    int8_t* codes;
    uint8_t* exps;
    int64_t ld, lde;
    int32_t vec;               // codes allow 8-element vectors
};

// ---- layer norm and the checkpoint passes (norm_kernels.hip) ----
struct NormArgs {
    const void* x;
    void* y;
    const void* gain;
    const void* bias;          // may be null
    float* mean;               // may be null
    float* rstd;               // may be null
    Act8View y8;               // codes null: none
    int64_t rows, ld_x, ld_y;
    int32_t cols;
    int32_t dt, pdt;           // 0 bf16, 1 f32: x and y; gain and bias
    int32_t vec;               // 16-byte vectors legal for x and y
    int32_t pvec;              // and for gain and bias
    float eps;
};

struct NormGradArgs {
    const void* dy;
    const void* x;
    const void* gain;
    const float* mean;
    const float* rstd;
    const void* add;           // may be null
    void* dx;
    void* dgain;
    void* dbias;               // may be null
    float* partial;            // [2][parts][cols] sums of dy xhat, then of dy
    int64_t rows, ld_dy, ld_x, ld_add, ld_dx;
    int32_t cols, parts;
    int32_t dt, pdt, vec, pvec, accumulate;
};

// Workgroups (= rows of the partial sums) of the backward pass.
int norm_grad_parts(int64_t rows, int cols);
// Whether the norm's launches can take so many rows.
bool norm_rows_fit(int64_t rows, int64_t cols);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);

struct Act8Args {
    const void* x;             // encode: source;  decode: unused
    void* y;                   // decode: destination
    Act8View q;
    int64_t rows, ld;
    int32_t cols, dt, vec;     // vec: 8-element vectors legal for x / y and codes
};
hipError_t launch_act8_encode(const Act8Args& a, hipStream_t s);
hipError_t launch_act8_decode(const Act8Args& a, hipStream_t s);

// ---- the linear layer's products (linear_kernels.hip) ----
enum LinKind : int { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };
enum LinAct : int { ACT_NONE = 0, ACT_GELU = 1, ACT_RELU_SQ = 2 };

// C (M x N) = A B over k.  A (m, k) at a[m * lda + k] (a_kc) or a[k * lda + m];
// B (n, k) at b[n * ldb + k] (b_kc) or b[k * ldb + n].
struct LinArgs {
    const void* a;
    const void* b;
    const uint8_t* a_exps;     // A is an 8-bit checkpoint (k x m codes): its exponents
    int64_t lda, ldb, lda_exps;
    int64_t M, N, K;
    int32_t dt;                // 0 bf16, 1 f32 (operands, and the tensors of the epilogue)
    int32_t a_kc, b_kc;
    int32_t a_dma, b_dma;      // 16-byte chunks of the operand are aligned and whole
    int32_t a8_vec;            // 8-element vectors legal for the codes
    int32_t kind, act;
    // epilogue: out = M x N, or N x M where out_trans
    void* out;
    int64_t ld_out;
    int32_t out_trans, out_dt, out_vec, accumulate;
    const void* bias;          // N, LIN_FWD
    int32_t bias_dt, bias_vec;
    const void* add;           // M x N: residual (LIN_FWD) or gradient to add (LIN_DX)
    int64_t ld_add;
    int32_t add_vec;
    void* z;                   // M x N: pre-activation, written (LIN_FWD) or read (LIN_DX)
    int64_t ld_z;
    int32_t z_vec;
    Act8View z8;               // or as an 8-bit checkpoint
    void* act_out;             // M x N: act(z) (LIN_DX)
    int64_t ld_act;
    int32_t act_vec;
    int32_t act_stream;        // act_out is stored past the L2s
    void* db;                  // N: column sums of B (LIN_DW), may be null
    int32_t db_dt;
    // split of the k range over workgroups: each writes its sums to `partial`
    // (float32, [splits][rows][cols] of the output's orientation, then
    // [splits][N] of the column sums) and a second kernel joins them
    int32_t splits;
    int32_t tile;              // tile edge: 64, 128 or 256
    int32_t deep;              // no more workgroups than CUs: more LDS stages
    float* partial;
    float* db_partial;
    // operands re-laid in the workspace before the product, as stored but with
    // aligned rows of a_ld / b_ld elements; 0: taken as they are
    void* a_ws;
    void* b_ws;
    int64_t a_ld, b_ld;
};

struct LinPlan {
    int tile = 128;
    int splits = 1;
    bool deep = false;
    int64_t a_ld = 0, b_ld = 0;
    size_t partial_bytes = 0, db_bytes = 0, a_bytes = 0, b_bytes = 0;
};
LinPlan plan_linear(const LinArgs& a);
hipError_t launch_linear(const LinArgs& a, hipStream_t s);

}  // namespace muon
