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
// Bytes bound it: of all the rows a lane reads T - 1 numbers of p and of q, and then one row of each.  A cluster takes a lane:
// its CTAs' warps sum tiles of the row, the CTAs put their sums into each other's shared memory, and a warp of the one that the
// threshold falls into finds the tile and reads that tile again.  256 lanes (a tenth padded) of 131072 with draft probabilities: 55 us,
// 4.4 TB/s; 256 lanes without them, or of one row, 48 us (2.8 TB/s); one lane 12 us a call.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kAcceptThreads = 256;  // of a CTA at most
constexpr int kAcceptBlock = 256;     // elements that a warp sums at a time: 8 a lane
constexpr int kAcceptTiles = 1024;    // tiles of a CTA's part of a row at most
constexpr int kAcceptMaxCluster = 8;

// a + b exactly, as a rounded sum and its error
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// r = max(p - q, 0) of one token as an exact pair; values that are not finite count as nothing
__device__ __forceinline__ float2 residual(float p, float q) {
    if (!(fabsf(p) <= FLT_MAX) || !(fabsf(q) <= FLT_MAX)) return make_float2(0.f, 0.f);
    const float s = p - q;
    const float2 r = make_float2(s, (p - s) - q);  // exact, since |p| >= |q|
    return p > q ? r : make_float2(0.f, 0.f);
}

struct RowPair {
    const float* p;
    const float* q;  // nullptr: q is 1 at `certain` and 0 elsewhere
    int certain;     // -1: nowhere
    __device__ __forceinline__ float2 at(int v) const {
        return residual(p[v], q != nullptr ? q[v] : (v == certain ? 1.f : 0.f));
    }
};

__device__ __forceinline__ double scan(double x, int lane) {  // inclusive, over the warp
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    return x;
}

// a pair's sum with another pair, to about 2^-46
__device__ __forceinline__ void add_pair(float2& a, float2 b) {
    const float2 s = two_sum(a.x, b.x);
    a = make_float2(s.x, s.y + (a.y + b.y));
}

// Two sums of max(p - q, 0) beside each other, each a pair of floats, with packed instructions (two tokens' share of each).
struct TwoSums {
    float2 hi = make_float2(0.f, 0.f), lo = make_float2(0.f, 0.f);
    __device__ __forceinline__ static float2 minus(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }  // rounded once
    __device__ __forceinline__ void add(float2 p, float2 q) {
        q = make_float2(fminf(p.x, q.x), fminf(p.y, q.y));  // nothing where q is the larger
        const float2 s = minus(p, q), e = minus(minus(p, s), q);  // exact, since |p| >= |q|
        const float2 t = __fadd2_rn(hi, s), u = minus(t, hi);
        lo = __fadd2_rn(lo, __fadd2_rn(__fadd2_rn(minus(hi, minus(t, u)), minus(s, u)), e));
        hi = t;
    }
    __device__ __forceinline__ float2 both() const {
        float2 a = make_float2(hi.x, lo.x);
        add_pair(a, make_float2(hi.y, lo.y));
        return a;
    }
};

__device__ __forceinline__ uint32_t shared_of(const void* p, uint32_t rank) {  // the same variable in another CTA of the cluster
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// tile: elements of a tile, a multiple of kAcceptBlock; CTA `rank` of the lane's cluster has tiles rank * per ..
__global__ void __launch_bounds__(kAcceptThreads) gdn_draft_accept_kernel(const DraftAcceptParams p, const int tile,
                                                                          const int per) {
    __shared__ float2 sums[kAcceptTiles];
    __shared__ double part[2][kAcceptMaxCluster];  // the CTAs' sums, of either pass
    __shared__ int sh_n;
    __shared__ bool sh_refused;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5, T = p.T, V = p.V;
    const int ncta = gridDim.x, rank = blockIdx.x, b = blockIdx.y;
    const int32_t* drafts = p.drafts + (int64_t)b * (T - 1);
    const int slot = p.indices != nullptr ? p.indices[b] : 0;
    const int x = warp == 0 && lane < T - 1 ? drafts[lane] : -1;  // asked for together with the slot
    const float u = warp == 0 && lane < T ? p.uniform[(int64_t)b * T + lane] : 0.f;
    if (slot < 0) {  // the whole cluster leaves
        if (slot < -1 && tid == 0 && rank == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
        return;
    }
    // shared memory of another CTA is there once that CTA runs: arrived at here, waited for before the first exchange
    if (ncta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const float* target = p.target + (int64_t)b * T * p.target_stride;
    const float* draft = p.draft != nullptr ? p.draft + (int64_t)b * (T - 1) * p.draft_stride : nullptr;
    if (warp == 0) {  // lane i: draft i
        bool good = false, real = false;
        if (lane < T - 1) {
            real = x >= 0 && x < V;
            if ((x < -1 || x >= V) && rank == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
            if (real) {
                const float px = target[lane * p.target_stride + x];
                const float qx = draft != nullptr ? draft[lane * p.draft_stride + x] : 1.f;
                good = (double)u * (double)qx < (double)px;
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
    const int tiles = (V + tile - 1) / tile, first = rank * per, mine = max(0, min(per, tiles - first));
    bool bad = false;
    double before = 0., total = 0., own = 0.;  // sums of the CTAs before this one, of all, of this one
    auto load = [&](int v0, int end, float (&pb)[8], float (&qb)[8]) {
        const float* pp = r.p + v0 + lane;
        const float* qq = r.q + v0 + lane;
        if (end - v0 >= kAcceptBlock) {  // a whole block: no bounds a number
#pragma unroll
            for (int i = 0; i < 8; ++i) pb[i] = pp[32 * i];
            if (r.q != nullptr)
#pragma unroll
                for (int i = 0; i < 8; ++i) qb[i] = qq[32 * i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = v0 + 32 * i + lane < end;
                pb[i] = in ? pp[32 * i] : 0.f;
                qb[i] = in && r.q != nullptr ? qq[32 * i] : 0.f;
            }
        }
        if (r.q == nullptr)
#pragma unroll
            for (int i = 0; i < 8; ++i) qb[i] = v0 + 32 * i + lane == r.certain ? 1.f : 0.f;
    };
    for (int pass = 0; pass < 2; ++pass) {
        // the warp's tiles, a block at a time, with the next block's loads in flight, be it of the same tile or of the next one
        int k = warp, v0 = 0, end = 0;
        float pv[8], qv[8];
        if (k < mine) {
            v0 = (first + k) * tile;
            end = V - v0 > tile ? v0 + tile : V;
            load(v0, end, pv, qv);
        }
        TwoSums acc;
        float2 probe = make_float2(0.f, 0.f);  // stays 0 while values are finite
        while (k < mine) {
            float pc[8], qc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) pc[i] = pv[i], qc[i] = qv[i];
            int k2 = k, v2 = v0, end2 = end;
            if (end - v0 > kAcceptBlock) {
                v2 += kAcceptBlock;
            } else if ((k2 += warps) < mine) {
                v2 = (first + k2) * tile;
                end2 = V - v2 > tile ? v2 + tile : V;
            }
            if (k2 < mine) load(v2, end2, pv, qv);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 p2 = make_float2(pc[i], pc[i + 1]), q2 = make_float2(qc[i], qc[i + 1]);
                probe = __ffma2_rn(q2, make_float2(0.f, 0.f), __ffma2_rn(p2, make_float2(0.f, 0.f), probe));
                acc.add(p2, q2);
            }
            if (k2 != k) {
                float2 sum = acc.both();
                if (!__all_sync(0xffffffffu, probe.x == 0.f && probe.y == 0.f)) {  // again, where a value that is not finite counts as nothing
                    bad = true;
                    sum = make_float2(0.f, 0.f);
                    for (int v = (first + k) * tile; v < end; v += min(kAcceptBlock, end - v)) {
                        load(v, end, pc, qc);
#pragma unroll
                        for (int i = 0; i < 8; ++i) add_pair(sum, residual(pc[i], qc[i]));
                    }
                }
#pragma unroll
                for (int m = 16; m >= 1; m >>= 1)
                    add_pair(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, m), __shfl_xor_sync(0xffffffffu, sum.y, m)));
                if (lane == 0) sums[k] = sum;
                acc = TwoSums();
                probe = make_float2(0.f, 0.f);
            }
            k = k2;
            v0 = v2;
            end = end2;
        }
        __syncthreads();
        // every warp forms the same sums, in the same order
        own = 0.;
        for (int k = lane; k < mine; k += 32) own += (double)sums[k].x + (double)sums[k].y;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) own += __shfl_xor_sync(0xffffffffu, own, m);
        before = 0.;
        total = own;
        if (ncta > 1) {  // every CTA puts its sum into every other's shared memory
            if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (tid < ncta)
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(shared_of(&part[pass][rank], (uint32_t)tid)), "d"(own)
                             : "memory");
            cluster_sync();
            total = 0.;
            for (int c = 0; c < ncta; ++c) {
                if (c == rank) before = total;
                total += part[pass][c];
            }
        }
        if (total > 0. || (r.q == nullptr && r.certain < 0)) break;
        r.q = nullptr;  // nothing is left of p - q: p itself
        r.certain = -1;
        __syncthreads();
    }
    if (__syncthreads_or(bad) && tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_NONFINITE);
    if (warp != 0) return;

    // The CTA whose part the threshold falls into draws the token: the first v whose running sum passes it.  Where rounding
    // leaves none, the last v with r_v > 0, which is in the last CTA with a sum.
    const double threshold = (double)__shfl_sync(0xffffffffu, u, T - 1) * total;
    bool writer = rank == 0, past = false;
    if (total > 0.) {
        int winner = 0;
        if (ncta > 1) {
            double upto = 0.;
            int found = -1, last = 0;
            for (int c = 0; c < ncta; ++c) {
                const double s = part[r.q == nullptr && r.certain < 0 && sh_refused ? 1 : 0][c];
                upto += s;
                if (s > 0.) last = c;
                if (found < 0 && s > 0. && upto > threshold) found = c;
            }
            past = found < 0;
            winner = past ? last : found;
        }
        writer = rank == winner;
    }
    if (!writer) return;
    int token = -1;
    if (total > 0.) {
        int found = -1, last = -1;
        for (int k0 = 0; k0 < mine && found < 0; k0 += 32) {
            const double s = k0 + lane < mine ? (double)sums[k0 + lane].x + (double)sums[k0 + lane].y : 0.;
            const double upto = before + scan(s, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, s > 0. && upto > threshold);
            const unsigned some = __ballot_sync(0xffffffffu, s > 0.);
            if (some != 0u) last = k0 + 31 - __clz(some);
            if (hit != 0u && !past) {
                found = k0 + __ffs(hit) - 1;
                before = __shfl_sync(0xffffffffu, upto - s, __ffs(hit) - 1);
            } else {
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (found < 0) past = true;
        const int k = first + (past ? last : found), end = min(V, (k + 1) * tile);
        for (int v0 = k * tile; v0 < end; v0 += kAcceptBlock) {  // 8 neighbours a lane
            float2 x[8];
            double s = 0.;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int v = v0 + 8 * lane + i;
                x[i] = v < end ? r.at(v) : make_float2(0.f, 0.f);
                s += (double)x[i].x + (double)x[i].y;
            }
            double upto = before + scan(s, lane) - s;
            int hit = INT32_MAX, some = -1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double own_i = (double)x[i].x + (double)x[i].y;
                upto += own_i;
                if (own_i > 0.) {
                    some = v0 + 8 * lane + i;
                    if (upto > threshold) hit = min(hit, some);
                }
            }
            some = __reduce_max_sync(0xffffffffu, some);
            hit = __reduce_min_sync(0xffffffffu, hit);
            if (some >= 0) token = some;  // the last so far
            if (!past && hit != INT32_MAX) {
                token = hit;
                break;
            }
            before = __shfl_sync(0xffffffffu, upto, 31);
        }
    } else if (lane == 0 && p.err != nullptr) {
        atomicOr(p.err, GDN_ERRBIT_NONFINITE);
    }
    if (lane == 0) p.accept_len[b] = n + 1;
    if (lane < T) p.tokens[(int64_t)b * T + lane] = lane < n ? x : lane == n ? token : -1;
}

}  // namespace

cudaError_t launch_draft_accept(const DraftAcceptParams& p, cudaStream_t s) {
    // Lanes that fill the GPU: CTAs of 128 threads, up to four a lane (two where those are six an SM), of which eight share an SM and some
    // read while others start, exchange and search.  Fewer lanes: 256 threads, as many CTAs as fill the GPU.  us in graph replays, the second
    // form / the first, with draft probabilities: 128 lanes of 131072 32.4 / 38.3, 160 47.6 / 42.1, 256 54.6 / 50.6; 128 of 32000 16.7 / 16.6,
    // 160 23.1 / 17.7, 256 23.5 / 21.2; 256 of 5000 12.1 / 9.5; without them: 128 of 131072 32.2 / 38.8, 160 44.8 / 41.7, 256 52.5 / 48.3
    // (of one row each 51.6 / 47.2).  Four CTAs a lane / two: 500 lanes of 32000 35.9 / 30.8, 464 of 131072 83.5 / 83.0.  (One lane of
    // 131072: 8 CTAs 15 us a call, 4 19, 2 27.)
    const int64_t sms = sm_count();
    const bool many = p.B >= sms;
    const int warps = many ? 4 : 8;
    int ncta = 1;
    if (many)
        while (ncta < 4 && p.V > ncta * 8192 && (int64_t)p.B * ncta < 6 * sms) ncta *= 2;
    else
        while (ncta < kAcceptMaxCluster && ((int64_t)p.V > (int64_t)ncta * 65536 || ((int64_t)p.B * ncta < 3 * sms && p.V > ncta * 2048))) ncta *= 2;
    // tiles of two blocks where a warp has more than eight blocks: its sum is formed once a tile (256 lanes of 131072: 59 us against 63)
    int tile = kAcceptBlock;
    if ((int64_t)p.V > (int64_t)tile * warps * ncta * 8) tile *= 2;
    while ((int64_t)tile * kAcceptTiles * ncta < p.V) tile *= 2;
    const int tiles = (p.V + tile - 1) / tile, per = (tiles + ncta - 1) / ncta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ncta, (unsigned)p.B);
    cfg.blockDim = dim3(32u * (unsigned)warps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ncta;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ncta > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, gdn_draft_accept_kernel, p, tile, per);
}

}  // namespace gdn
