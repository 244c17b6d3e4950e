// qat_few.h -- binary32 products of a few tokens (internal; not part of the C
// ABI).  All matrices are row-major without padding, 16-byte aligned.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qat.h"
#include "qat_launch.h"

namespace qat {

// fp32 layers of this many tokens or fewer take these kernels (both sides' times, and
// where the limit loses, in kernels_few.cu)
constexpr int64_t kFewTokens = 32;

// h[t, f] = act(x wg^T) * (x wu^T); g and u kept where gp is set
qat_status launch_few_gated(const float* x, int64_t t, int64_t d, int64_t f, const float* wg,
                            const float* wu, int act, float* h, float* gp, float* up, bool pdl,
                            cudaStream_t s);
// out[t, n] = a[t, k] w[n, k]^T
qat_status launch_few_rows(const float* a, int64_t t, int64_t k, int64_t n, const float* w,
                           float* out, bool pdl, cudaStream_t s);
// dh = dy[t, d] wd[d, f]; dg = dh * up * act'(gp), du = dh * act(gp)
qat_status launch_few_gated_bwd(const float* dy, int64_t t, int64_t d, int64_t f, const float* wd,
                                int act, const float* gp, const float* up, float* dg, float* du,
                                bool pdl, cudaStream_t s);
// out[t, n] = a[t, k] wa[k, n] + b[t, k] wb[k, n]
qat_status launch_few_cols2(const float* a, const float* b, int64_t t, int64_t k, int64_t n,
                            const float* wa, const float* wb, float* out, bool pdl, cudaStream_t s);

}  // namespace qat
