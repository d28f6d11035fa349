// iabn_block_internal.h -- host-side types shared by the entry points of
// iabn_block.h and the kernels behind them.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace iabn {

// Columns that share one checkpoint scale (IABN_Q8_GROUP).
constexpr int kQGroup = 128;

enum : int { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
enum : int { kNoCodes = -1, kE4M3 = 0, kInt8 = 1 };
enum : int { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

inline int64_t q_groups(int64_t cols) { return (cols + kQGroup - 1) / kQGroup; }

struct BlockFwd {
    const void* u;   // null: norm of h alone
    const void* h;
    void* h_out;
    void* n;
    const float *gamma_post, *beta_post, *gate, *gamma_pre, *beta_pre;
    float *mean_post, *rstd_post, *mean_pre, *rstd_pre;
    uint8_t *q_post, *q_pre;
    float *scale_post, *scale_pre;
    int64_t rows, rows_per_gate;
    int cols, groups;
    int post, pre, format;
    float alpha, eps_post, eps_pre;
};

struct BlockBwd {
    const void* su;   // u, or the codes of uhat; null where uhat is not needed
    const void* sh;   // h_out, or the codes of xhat; null with pre = none
    const float *scale_post, *scale_pre;   // of codes
    const void* dh_out;
    const void* dn;
    void* dh;
    void* du;
    const float *gamma_post, *beta_post, *gate, *gamma_pre;
    const float *mean_post, *rstd_post, *mean_pre, *rstd_pre;
    float *dgamma_post, *dbeta_post, *dgate, *dgamma_pre, *dbeta_pre;
    float* work;   // partial sums
    int64_t rows, rows_per_gate;
    int64_t gates;   // gate rows (1 without a gate)
    int64_t workers; // blocks (clusters) of the row pass
    int cols, groups;
    int post, pre, format;
    float alpha;
};

// Workers of the backward's row pass (a block or a cluster of them; laid out for
// 148 SMs), and the partial-sum rows of `cols` floats they need: two a worker
// (dn*xhat, dn) and two a (worker, gate row) pair
// (t*uhat, t), the pair (w, g) in slot w + g: workers take consecutive rows,
// so from pair to pair at least one of the two grows.
int64_t block_bwd_workers(int64_t rows, int64_t cols);
__host__ __device__ inline int64_t block_bwd_slots(int64_t workers, int64_t gates) { return workers + gates; }

struct Gated {
    const void *a, *b;           // inputs, or
    const uint8_t *qa, *qb;      // their codes (backward)
    uint8_t *qa_out, *qb_out;    // forward: codes written, or null
    float *sa_out, *sb_out;
    const float *sa, *sb;
    const void* dz;
    void *z, *da, *db;
    int64_t rows, cols, ld, ld_grad;
    int act, format;
};

struct Check8 {
    const void* x;
    void* y;
    uint8_t* q;
    float* scale;
    const float *gamma, *beta;
    int64_t rows, cols, ld;
    int format;
};

cudaError_t block_forward(const BlockFwd& a, int dtype, cudaStream_t s, int sms);
cudaError_t block_backward(const BlockBwd& a, int dtype, bool codes, cudaStream_t s, int sms);
cudaError_t gated_forward(const Gated& a, int dtype, cudaStream_t s, int sms);
cudaError_t gated_backward(const Gated& a, int dtype, bool codes, cudaStream_t s, int sms);
cudaError_t check8_store(const Check8& a, int dtype, cudaStream_t s, int sms);
cudaError_t check8_load(const Check8& a, int dtype, cudaStream_t s, int sms);

}  // namespace iabn
