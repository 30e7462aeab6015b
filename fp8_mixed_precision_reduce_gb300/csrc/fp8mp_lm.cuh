// fp8mp_lm.cuh -- launchers of the kernels around the FP8 blocks of a language model.
// Not part of the ABI.
#pragma once

#include "fp8mp_internal.cuh"

namespace fp8mp {

// The norm (norm.cu; M, K > 0, but M == 0 for the weight's gradient alone), the
// log probabilities (logprob.cu; M > 0) and the embedding (embed.cu; K > 0, M > 0
// forward, V > 0 backward; table_kind: 0 E4M3, 1 bf16, 2 fp32); arguments validated.
int64_t rmsnorm_workspace_bytes(int64_t M, int64_t K);
int launch_rmsnorm_fwd(const void *x, int x_dtype, const void *r, void *t, int r_dtype, int64_t M, int64_t K,
                       const void *w, int w_dtype, float eps, const float *y_scale, void *y, int y_dtype,
                       float *y_amax, float *rstd, cudaStream_t s, const DeviceInfo &dev);
int launch_rmsnorm_bwd(const void *dy, int dy_dtype, const void *dtotal, const void *t, int t_dtype, const float *rstd,
                       int64_t M, int64_t K, const void *w, int w_dtype, void *dr, void *dx, void *dw, int dw_dtype,
                       void *workspace, cudaStream_t s, const DeviceInfo &dev);
int launch_logprobs_fwd(const void *x, int x_dtype, int64_t M, int64_t V, int64_t ld, const int64_t *target,
                        float *logprob, float *stats, float *entropy, float *top, int64_t *ids, int k, cudaStream_t s,
                        const DeviceInfo &dev);
int launch_logprobs_bwd(const void *x, int x_dtype, int64_t M, int64_t V, int64_t ld, const int64_t *target,
                        const float *stats, const float *dlogprob, const float *entropy, const float *dentropy,
                        const float *scale, void *dlogits, float *amax, cudaStream_t s, const DeviceInfo &dev);
int64_t embedding_workspace_bytes(int64_t M, int64_t K);
int launch_embedding_fwd(const int64_t *ids, int64_t M, const void *table, int table_kind, int64_t V, int64_t K,
                         const float *sinv, float scale, void *out, int out_dtype, cudaStream_t s, const DeviceInfo &dev);
int launch_embedding_bwd(const int64_t *ids, int64_t M, const void *dy, int dy_dtype, int64_t V, int64_t K, float scale,
                         void *dtable, int out_dtype, void *workspace, cudaStream_t s, const DeviceInfo &dev);

}  // namespace fp8mp
