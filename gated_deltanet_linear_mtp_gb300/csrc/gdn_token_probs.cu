// gdn_token_probs.cu -- token probabilities of logits rows with a temperature for each lane (sm_103a):
//     p_v = exp((x_v - max x) / T) / sum_u exp((x_u - max x) / T)
// for row r = (lane, token); T = 0 (or below the smallest normal number) puts 1 at the first of the largest logits.
//
// -inf logits (forbidden tokens) get 0; a row of nothing else gets zeros.  A NaN or +inf logit, or a temperature that is
// negative or not finite, makes the row zeros and sets GDN_ERRBIT_NONFINITE.
//
// Bytes bound it: a row is read once from DRAM and written once (512 rows of 131072 bf16 74 us, 5.4 TB/s, of 32000 16; 256 of 131072 fp32 56 us,
// 4.8 TB/s; one row of 50001 fp32 6.8 us a call).  A thread-block cluster takes a row, each CTA a run of it:
// a first pass with the running maximum and sum, 8 or 16 numbers at a time, one exchange of (maximum, sum, index) within the
// cluster, and a second pass that reads the run again (from L1 or L2, where it still is) and writes.
//
// exp((x - m) / T) = 2^(c x - o), c = log2(e) / T and o = c m rounded: one multiply-add that rounds its result alone, and a
// common error of o that the division by the sum takes out again.  ex2.approx.ftz adds 2^-22 and takes what is below 2^-126 as 0.
// That needs |o| <= 2^20 (o's error stays below 1/16): a row whose largest logit lies beyond, one with NaN or +inf, and one
// whose largest entries are the type's lowest value go through the first pass again with differences x - m, and checks.  NaN is no
// maximum, so the sum alone carries it: also that of a thread, warp or CTA which has met nothing but NaN and -inf.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "gdn.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kProbMaxCluster = 8;

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes of logits as numbers
__device__ __forceinline__ void unpack16(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack16(const uint4& r, float (&f)[8]) {  // bf16: element 2i in the lower half of word i
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// four logits
template <typename InT>
using Four = typename std::conditional<sizeof(InT) == 2, uint2, float4>::type;
__device__ __forceinline__ float4 as_f32(const float4& r) { return r; }
__device__ __forceinline__ float4 as_f32(const uint2& r) {
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// what a part of a row has: its largest logit, the sum against it, the place of the first largest, and whether it is not sound
struct Part {
    float m, s;
    int at, bad;
};

// Weights of a row.  kFar: from differences to the maximum, for logits of any size; else from c x - o.
template <bool kFar>
struct Weights {
    float c;
    __device__ __forceinline__ float offset(float m) const { return kFar ? m : fmaxf(c * m, -1048576.f); }
    __device__ __forceinline__ float operator()(float x, float o) const {
        if (!kFar) return ex2(fmaf(c, x, -o));
        const float d = x - o;  // -inf where x is, or where it lies that far below
        return d > -FLT_MAX ? ex2(c * d) : 0.f;
    }
    __device__ __forceinline__ float ratio(float o, float o2) const {  // of the weights against o to those against o2 >= o
        return kFar ? (*this)(o, o2) : ex2(o - o2);
    }
    // the parts of N neighbouring lanes as one: the largest first, then every sum against it (o: the offset of a's)
    template <int N>
    __device__ __forceinline__ Part joined(Part a, float o) const {
        float m = a.m;
#pragma unroll
        for (int k = N / 2; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        float s = a.m > -INFINITY ? a.s * ratio(o, offset(m)) : a.s;  // without a maximum: 0, or NaN, which stays
        int at = a.m == m ? a.at : INT32_MAX;
#pragma unroll
        for (int k = N / 2; k >= 1; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        return Part{m, s, __reduce_min_sync(0xffffffffu, at), __any_sync(0xffffffffu, a.bad)};
    }
    // the parts of a cluster as one, in every thread
    __device__ __forceinline__ Part of_cluster(const Part* parts, int n) const {
        const int i = threadIdx.x & 7;
        const Part a = i < n ? parts[i] : Part{-INFINITY, 0.f, INT32_MAX, 0};
        return joined<8>(a, offset(a.m));
    }
};

__device__ __forceinline__ uint32_t shared_of(const void* p, uint32_t rank) {  // the same variable in another CTA of the cluster
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

// one thread's part of a row
template <bool kFar>
struct Sum {
    const Weights<kFar> w;
    float m = -INFINITY, o = 0.f, s = 0.f;
    int at = INT32_MAX;
    bool bad = false;
    __device__ __forceinline__ void raise(float top) {  // a new maximum
        const float o2 = w.offset(top);
        s = m > -INFINITY ? s * w.ratio(o, o2) : s;  // 0 before the first logit above -inf, or NaN, which stays
        m = top;
        o = o2;
    }
    template <int E>
    __device__ __forceinline__ void take(const float (&f)[E], int v, bool greedy) {  // logits v .. v + E - 1
        float top = f[0];
#pragma unroll
        for (int i = 1; i < E; ++i) top = fmaxf(top, f[i]);
        if (top > m) {
            raise(top);
            if (greedy)
#pragma unroll
                for (int i = E - 1; i >= 0; --i)
                    if (f[i] == top) at = v + i;
        }
        if (kFar)
#pragma unroll
            for (int i = 0; i < E; ++i) bad |= !(f[i] <= FLT_MAX);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            s0 += w(f[i], o);
            s1 += w(f[i + 1], o);
        }
        s += s0 + s1;
    }
    __device__ __forceinline__ void take_one(float f, int v) {
        if (f == m) at = min(at, v);
        if (f > m) {
            raise(f);
            at = v;
        }
        bad |= kFar && !(f <= FLT_MAX);
        s += w(f, o);
    }
    // the CTA's part, in every thread
    __device__ __forceinline__ Part of_cta(Part* warps) const {
        const int lane = threadIdx.x & 31;
        const Part all = w.template joined<32>(Part{m, s, at, bad}, o);
        if (lane == 0) warps[threadIdx.x >> 5] = all;
        __syncthreads();
        const Part mine = warps[lane % kProbWarps];
        return w.template joined<kProbWarps>(mine, w.offset(mine.m));
    }
};

__device__ __forceinline__ void put_part(uint32_t to, const Part& a) {  // into a CTA of the cluster
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(__float_as_uint(a.m)), "r"(__float_as_uint(a.s)),
                 "r"(a.at), "r"(a.bad)
                 : "memory");
}

// A CTA's run of a row: elements lo .. hi - 1, of them whole 16-byte pieces a .. b - 1 (by their addresses)
template <typename InT>
struct RunOf {
    static constexpr int EPC = 16 / sizeof(InT);
    int lo, hi, a, b;
    __device__ __forceinline__ RunOf(const InT* x, int V, int rank, int run) {
        lo = (int)min((int64_t)rank * run, (int64_t)V);
        hi = (int)min((int64_t)lo + run, (int64_t)V);
        const int off = (int)((reinterpret_cast<uintptr_t>(x + lo) & 15u) / sizeof(InT));
        a = min(hi, lo + (off == 0 ? 0 : EPC - off));
        b = a + (hi - a) / EPC * EPC;
    }
    __device__ __forceinline__ int pieces() const { return (b - a) / EPC; }
    __device__ __forceinline__ int edge() const { return (a - lo) + (hi - b); }  // elements in no piece
    __device__ __forceinline__ int edge_at(int i) const { return i < a - lo ? lo + i : b + i - (a - lo); }
};

// Pieces in flight a thread and CTAs an SM: two and four for bf16, four and three for fp32 (us the other way about: 512 rows of 65536 bf16 42.7
// against 39.8, 256 of 131072 fp32 61.5 against 58.3; CTAs of 256 and 1024 threads were slower).
// Tried for rows of 131072: the run kept in registers between the passes (one exp an element, fewer threads in flight: 158 us then), the
// maximum first and the sum after it, and a persistent cluster whose next run lands in shared memory meanwhile (104 us).
template <typename InT>
__global__ void __launch_bounds__(kProbThreads, sizeof(InT) == 2 ? 4 : 3) gdn_token_probs_kernel(const TokenProbsParams p, const int run) {
    constexpr int EPC = 16 / sizeof(InT);  // elements of a 16-byte piece
    constexpr int U = 16 / EPC;            // pieces in flight a thread
    __shared__ Part warps[2][kProbWarps];  // of the first pass, and of its repetition
    __shared__ Part parts[2][kProbMaxCluster];
    const int tid = threadIdx.x;
    const int ncta = gridDim.x, rank = blockIdx.x;  // the cluster is the grid's x
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= (int64_t)p.B * p.T) return;  // the whole cluster leaves
    // shared memory of another CTA is there once that CTA runs: arrived at here, waited for before the exchange
    if (ncta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const InT* x = static_cast<const InT*>(p.logits) + row * p.logits_stride;
    float* y = p.probs + row * p.probs_stride;
    const float T = p.temperature[row / p.T];
    const bool greedy = T >= 0.f && T < FLT_MIN;
    const float c = 1.44269504f / (greedy ? 1.f : T);
    const RunOf<InT> r(x, p.V, rank, run);
    const int lo = r.lo, hi = r.hi, a = r.a, pieces = r.pieces(), edge = r.edge();
    const uint4* xv = reinterpret_cast<const uint4*>(x + a);

    auto first_pass = [&](auto wf) -> Part {
        constexpr bool kFar = sizeof(wf) != sizeof(float);
        const Weights<kFar> w{c};
        Sum<kFar> sum{w};
        for (int c0 = tid; c0 < pieces; c0 += U * kProbThreads) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * kProbThreads < pieces) raw[u] = xv[c0 + u * kProbThreads];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u * kProbThreads >= pieces) break;
                float f[EPC];
                unpack16(raw[u], f);
                sum.take(f, a + (c0 + u * kProbThreads) * EPC, greedy);
            }
        }
        if (tid < edge) sum.take_one(as_f32(x[r.edge_at(tid)]), r.edge_at(tid));
        Part all = sum.of_cta(warps[kFar]);
        if (ncta > 1) {  // every CTA puts its part into every other's shared memory
            if (!kFar) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (tid < ncta) put_part(shared_of(&parts[kFar][rank], (uint32_t)tid), all);
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            all = w.of_cluster(parts[kFar], ncta);
        }
        return all;
    };
    Part all = first_pass(float{});
    // every thread of the cluster has the same sums, and takes the same way
    const bool far = !(fabsf(c * all.m) <= 1048576.f) || !(all.s > 0.f && all.s <= FLT_MAX);
    if (far && all.m != -INFINITY) all = first_pass(double{});
    all.bad |= !(T >= 0.f) || T > FLT_MAX || !(all.s <= FLT_MAX);
    if (all.bad && tid == 0 && rank == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_NONFINITE);
    const bool none = all.bad || !(all.m > -INFINITY);
    if (none || greedy) {  // zeros, and a 1 at the place of the first largest
        for (int v = lo + tid; v < hi; v += kProbThreads) y[v] = !none && v == all.at ? 1.f : 0.f;
        return;
    }
    auto second_pass = [&](auto wf) {
        const Weights<sizeof(wf) != sizeof(float)> w{c};
        const float o = w.offset(all.m), f = 1.f / all.s;
        if ((reinterpret_cast<uintptr_t>(y + a) & 15u) == 0) {
            // four numbers a thread and store: a warp writes whole lines (eight as two stores leave half sectors: 98 us against 75)
            const Four<InT>* x4 = reinterpret_cast<const Four<InT>*>(x + a);
            const int fours = pieces * (EPC / 4);
            constexpr int U4 = U * EPC / 4;
            for (int c0 = tid; c0 < fours; c0 += U4 * kProbThreads) {
                Four<InT> raw[U4];
#pragma unroll
                for (int u = 0; u < U4; ++u)
                    if (c0 + u * kProbThreads < fours) raw[u] = x4[c0 + u * kProbThreads];
#pragma unroll
                for (int u = 0; u < U4; ++u) {
                    if (c0 + u * kProbThreads >= fours) break;
                    const float4 e = as_f32(raw[u]);
                    __stcs(reinterpret_cast<float4*>(y + a) + c0 + u * kProbThreads,
                           make_float4(w(e.x, o) * f, w(e.y, o) * f, w(e.z, o) * f, w(e.w, o) * f));
                }
            }
            if (tid < edge) y[r.edge_at(tid)] = w(as_f32(x[r.edge_at(tid)]), o) * f;
        } else {  // the places of x and y differ: neighbours a warp
            for (int v0 = lo + tid; v0 < hi; v0 += 8 * kProbThreads) {
                InT raw[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (v0 + u * kProbThreads < hi) raw[u] = x[v0 + u * kProbThreads];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (v0 + u * kProbThreads < hi) __stcs(y + v0 + u * kProbThreads, w(as_f32(raw[u]), o) * f);
            }
        }
    };
    if (far)
        second_pass(double{});
    else
        second_pass(float{});
}

template <typename InT>
cudaError_t launch_t(const TokenProbsParams& p, cudaStream_t s) {
    const int64_t rows = (int64_t)p.B * p.T;
    // CTAs a row.  Runs of up to 32768 elements where rows fill the GPU (512 rows of 131072 bf16: 4 CTAs 75 us, 2 81, 8 87; of 32768:
    // 1 CTA 19 us, 2 23, 4 30: a CTA's start and the exchange cost some microseconds), of 4096 where they do not (one row of 131072:
    // 8 CTAs 6.7 us, 4 8.7, 1 20.5)
    const int sms = sm_count();
    int ncta = 1;
    while (ncta < kProbMaxCluster && ((int64_t)p.V > (int64_t)ncta * 32768 || (rows * ncta < sms && p.V > ncta * 4096))) ncta *= 2;
    const int run = (int)(((int64_t)p.V + ncta * 64 - 1) / (ncta * 64) * 64);
    const unsigned gy = (unsigned)(rows < 65535 ? rows : 65535);  // rows < 2^31: z stays below 2^16
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ncta, gy, (unsigned)((rows + gy - 1) / gy));
    cfg.blockDim = dim3(kProbThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ncta;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ncta > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, gdn_token_probs_kernel<InT>, p, run);
}

}  // namespace

cudaError_t launch_token_probs(const TokenProbsParams& p, cudaStream_t s) {
    return p.bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace gdn
