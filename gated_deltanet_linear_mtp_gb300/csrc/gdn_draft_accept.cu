// gdn_draft_accept.cu -- acceptance of drafted tokens against the target's probabilities, and the token after them (sm_103a).
//
// Lane b has T rows of target probabilities p_0 .. p_{T-1}, T - 1 drafts x_i with the probabilities q_i they were drawn from, and
// T numbers u_i in [0, 1).  Draft i is accepted while u_i q_i(x_i) < p_i(x_i); with a drafts accepted, the next token is drawn
// from row a: r = max(p_a - q_a, 0) if draft a was refused (p_a if that leaves nothing, or after the last draft), at the first
// v with r_v > 0 and r_0 + .. + r_v > u_{T-1} sum r.
//
// A token is a whole number, so the sums must be right wherever the threshold falls, next to the border of two tokens of a
// vocabulary of 2^17 too: p - q is taken exactly (as a pair of floats) and summed in pairs of floats (about 2^-46 of the sum, where
// 64-bit additions of every element would take longer than the reads), the sums of tiles and the search inside one in 64 bits.
//
// Bytes bound it: of all the rows a lane reads T - 1 numbers of p and of q, and then one row of each.  One CTA a lane: its
// warps sum tiles of the row, one warp finds the tile that the threshold falls into and searches that tile again.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kAcceptThreads = 512;
constexpr int kAcceptWarps = kAcceptThreads / 32;
constexpr int kAcceptTiles = 1024;  // tiles of a row at most

// a + b exactly, as a rounded sum and its error
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// r = max(p - q, 0) of one token as an exact pair; values that are not finite count as nothing
__device__ __forceinline__ float2 residual(float p, float q, bool& bad) {
    if (!(fabsf(p) <= FLT_MAX) || !(fabsf(q) <= FLT_MAX)) {
        bad = true;
        return make_float2(0.f, 0.f);
    }
    return p > q ? two_sum(p, -q) : make_float2(0.f, 0.f);
}

struct RowPair {
    const float* p;
    const float* q;  // nullptr: q is 1 at `certain` and 0 elsewhere
    int certain;     // -1: nowhere
    __device__ __forceinline__ float2 at(int v, bool& bad) const {
        return residual(p[v], q != nullptr ? q[v] : (v == certain ? 1.f : 0.f), bad);
    }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

__global__ void __launch_bounds__(kAcceptThreads) gdn_draft_accept_kernel(const DraftAcceptParams p, const int tile) {
    __shared__ double sums[kAcceptTiles];
    __shared__ int sh_n;
    __shared__ bool sh_refused;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x, T = p.T, V = p.V;
    if (p.indices != nullptr) {
        const int slot = p.indices[b];
        if (slot == -1) return;
        if (slot < -1) {
            if (tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
            return;
        }
    }
    const int32_t* drafts = p.drafts + (int64_t)b * (T - 1);
    const float* target = p.target + (int64_t)b * T * p.target_stride;
    const float* draft = p.draft != nullptr ? p.draft + (int64_t)b * (T - 1) * p.draft_stride : nullptr;
    if (warp == 0) {  // lane i: draft i
        bool good = false, real = false;
        if (lane < T - 1) {
            const int x = drafts[lane];
            real = x >= 0 && x < V;
            if (x < -1 || x >= V) {
                if (p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
            }
            if (real) {
                const float px = target[lane * p.target_stride + x];
                const float qx = draft != nullptr ? draft[lane * p.draft_stride + x] : 1.f;
                good = (double)p.uniform[(int64_t)b * T + lane] * (double)qx < (double)px;
            }
        }
        const unsigned goods = __ballot_sync(0xffffffffu, good), reals = __ballot_sync(0xffffffffu, real);
        if (lane == 0) {
            const int n = __ffs(~goods) - 1;  // lanes past the drafts are not good: n <= T - 1
            sh_n = n;
            sh_refused = (reals >> n) & 1u;
        }
    }
    __syncthreads();
    const int n = sh_n;
    RowPair r{target + n * p.target_stride, nullptr, -1};
    if (sh_refused) {
        if (draft != nullptr)
            r.q = draft + n * p.draft_stride;
        else
            r.certain = drafts[n];
    }
    const int tiles = (V + tile - 1) / tile;
    bool bad = false;
    double total = 0.;
    for (int pass = 0; pass < 2; ++pass) {
        for (int k = warp; k < tiles; k += kAcceptWarps) {
            float hi = 0.f, lo = 0.f;
            const int end = min(V, (k + 1) * tile);
            for (int v = k * tile + lane; v < end; v += 32) {
                const float2 x = r.at(v, bad);
                const float2 s = two_sum(hi, x.x);
                hi = s.x;
                lo += s.y + x.y;
            }
            const double sum = warp_sum((double)hi + (double)lo);
            if (lane == 0) sums[k] = sum;
        }
        __syncthreads();
        total = 0.;
        for (int k = lane; k < tiles; k += 32) total += sums[k];
        total = warp_sum(total);
        if (total > 0. || (r.q == nullptr && r.certain < 0)) break;
        r.q = nullptr;  // nothing is left of p - q: p itself
        r.certain = -1;
        __syncthreads();
    }
    if (__syncthreads_or(bad) && tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_NONFINITE);
    if (warp != 0) return;

    // the first v whose running sum passes the threshold; where rounding leaves none, the last v with r_v > 0
    const double threshold = (double)p.uniform[(int64_t)b * T + T - 1] * total;
    double before = 0.;
    int token = -1;
    if (total > 0.) {
        int found = -1, last = -1;
        for (int k0 = 0; k0 < tiles && found < 0; k0 += 32) {
            const double own = k0 + lane < tiles ? sums[k0 + lane] : 0.;
            double upto = own;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, upto, m);
                if (lane >= m) upto += y;
            }
            upto += before;
            const unsigned hit = __ballot_sync(0xffffffffu, own > 0. && upto > threshold);
            const unsigned some = __ballot_sync(0xffffffffu, own > 0.);
            if (some != 0u) last = k0 + 31 - __clz(some);
            if (hit != 0u) {
                found = k0 + __ffs(hit) - 1;
                before = __shfl_sync(0xffffffffu, upto - own, __ffs(hit) - 1);
            } else {
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        const bool past = found < 0;
        const int k = past ? last : found;
        const int end = min(V, (k + 1) * tile);
        bool dummy = false;
        for (int v0 = k * tile; v0 < end; v0 += 32) {
            const float2 x = v0 + lane < end ? r.at(v0 + lane, dummy) : make_float2(0.f, 0.f);
            const double own = (double)x.x + (double)x.y;
            double upto = own;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, upto, m);
                if (lane >= m) upto += y;
            }
            upto += before;
            const unsigned hit = __ballot_sync(0xffffffffu, own > 0. && upto > threshold);
            const unsigned some = __ballot_sync(0xffffffffu, own > 0.);
            if (some != 0u) token = v0 + 31 - __clz(some);  // the last so far
            if (!past && hit != 0u) {
                token = v0 + __ffs(hit) - 1;
                break;
            }
            before = __shfl_sync(0xffffffffu, upto, 31);
        }
    } else if (lane == 0 && p.err != nullptr) {
        atomicOr(p.err, GDN_ERRBIT_NONFINITE);
    }
    if (lane == 0) p.accept_len[b] = n + 1;
    if (lane < T) p.tokens[(int64_t)b * T + lane] = lane < n ? drafts[lane] : lane == n ? token : -1;
}

}  // namespace

cudaError_t launch_draft_accept(const DraftAcceptParams& p, cudaStream_t s) {
    int tile = 256;
    while ((int64_t)tile * kAcceptTiles < p.V) tile *= 2;
    gdn_draft_accept_kernel<<<p.B, kAcceptThreads, 0, s>>>(p, tile);
    return cudaGetLastError();
}

}  // namespace gdn
