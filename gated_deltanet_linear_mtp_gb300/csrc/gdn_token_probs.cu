// gdn_token_probs.cu -- token probabilities of logits rows with a temperature for each lane (sm_103a):
//     p_v = exp((x_v - max x) / T) / sum_u exp((x_u - max x) / T)
// for row r = (lane, token); T = 0 (or below the smallest normal number) puts 1 at the first of the largest logits.
//
// -inf logits (forbidden tokens) get 0; a row of nothing else gets zeros.  A NaN or +inf logit, or a temperature that is
// negative or not finite, makes the row zeros and sets GDN_ERRBIT_NONFINITE.
//
// Bytes bound it: a row is read once from DRAM and written once.  A CTA takes a row: a first pass with the running maximum
// and sum, a second over the row again (from L2) that writes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// (x - top) / T: the quotient to within one rounding from the reciprocal and one correction
__device__ __forceinline__ float over_t(float d, float T, float rT) {
    const float q = d * rT;
    return fmaf(fmaf(-q, T, d), rT, q);
}

__device__ __forceinline__ float weight(float x, float top, float T, float rT) {
    const float d = x - top;
    // below e^-104 fp32 has nothing left; d may be -inf, whose quotient is not formed
    return d * rT < -104.f ? 0.f : expf(over_t(d, T, rT));
}

template <typename InT>
__global__ void __launch_bounds__(kProbThreads) gdn_token_probs_kernel(const TokenProbsParams p) {
    __shared__ float sh_m[kProbWarps], sh_s[kProbWarps];
    __shared__ int sh_i[kProbWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x;
    const InT* x = static_cast<const InT*>(p.logits) + row * p.logits_stride;
    float* y = p.probs + row * p.probs_stride;
    const float T = p.temperature[row / p.T];
    const bool greedy = T >= 0.f && T < FLT_MIN;
    const float rT = greedy ? 1.f : 1.f / T;
    bool bad = !(T >= 0.f) || T > FLT_MAX;

    float m = -INFINITY, s = 0.f;
    int at = p.V;
    for (int i = tid; i < p.V; i += kProbThreads) {
        const float f = as_f32(x[i]);
        bad |= !(f <= FLT_MAX);
        if (f > m) {
            if (m > -INFINITY) s *= weight(m, f, T, rT);
            m = f;
            at = i;
        }
        if (m > -INFINITY) s += weight(f, m, T, rT);
    }
    bad = __syncthreads_or(bad);
    auto join = [&](float m2, float s2, int at2) {
        const float t = fmaxf(m, m2);
        if (t > -INFINITY && !bad && !greedy) s = (s > 0.f ? s * weight(m, t, T, rT) : 0.f) + (s2 > 0.f ? s2 * weight(m2, t, T, rT) : 0.f);
        at = m2 > m || (m2 == m && at2 < at) ? at2 : at;
        m = t;
    };
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, k), s2 = __shfl_xor_sync(0xffffffffu, s, k);
        join(m2, s2, __shfl_xor_sync(0xffffffffu, at, k));
    }
    if (lane == 0) sh_m[warp] = m, sh_s[warp] = s, sh_i[warp] = at;
    __syncthreads();
    m = sh_m[lane % kProbWarps], s = sh_s[lane % kProbWarps], at = sh_i[lane % kProbWarps];
#pragma unroll
    for (int k = 1; k < kProbWarps; k <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, k), s2 = __shfl_xor_sync(0xffffffffu, s, k);
        join(m2, s2, __shfl_xor_sync(0xffffffffu, at, k));
    }
    if (bad && tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_NONFINITE);
    const bool none = bad || !(m > -INFINITY);
    const float rs = none ? 0.f : 1.f / s;
    for (int i = tid; i < p.V; i += kProbThreads) {
        float f = 0.f;
        if (greedy)
            f = !none && i == at ? 1.f : 0.f;
        else if (!none)
            f = weight(as_f32(x[i]), m, T, rT) * rs;
        y[i] = f;
    }
}

}  // namespace

cudaError_t launch_token_probs(const TokenProbsParams& p, cudaStream_t s) {
    const unsigned rows = (unsigned)(p.B * p.T);
    if (p.bf16)
        gdn_token_probs_kernel<__nv_bfloat16><<<rows, kProbThreads, 0, s>>>(p);
    else
        gdn_token_probs_kernel<float><<<rows, kProbThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
