// gdn_page_plan.cu -- block tables, slot map, positions and offsets of one step's tokens from the lanes' lengths.
//
//     need_b = max(0, ceil((kv_len_b + new_b) / P) - held_b)        pages lane b still wants
//     upto_b = need_0 + .. + need_b;  lane b gets them (in this order) while taken + upto_b <= the free list's length
//     table[b, held_b + i] = free_pages[taken + upto_b - need_b + i]
//     slot(token at position x of lane b) = table[b, x / P] * P + x % P
//
// Latency bound: a step's lengths and tokens are a few KB to a few MB.  So one launch does everything: every CTA scans
// all lanes' lengths by itself (B values from L2; cheaper than a second launch or a wait between CTAs) and then writes
// its own slice of the tables and of the tokens, finding a token's lane by binary search in shared memory.  A
// new page is taken from the free list directly, so no CTA reads what another one writes; held and taken, which the
// caller may update in place, are written by the last CTA to finish, after all have read them.  Measured: 256 lanes of 8 new
// tokens 8.6 us, 64 prompts of 256 .. 4096 tokens (pages of 16) 10.5 us, where an empty launch takes about 4 (10.6 us for the
// former with one token of a thread at a time and a warp a lane for the new pages).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "gdn_common.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 512;
constexpr size_t smem_bytes(int lanes) { return ((size_t)5 * lanes + 1) * 4; }

struct LaneNeed {
    int64_t add;   // tokens this lane has in the packed order
    int64_t need;  // pages it wants
    bool ok;       // its lengths are in range
};

__device__ __forceinline__ LaneNeed lane_need(const PagePlanParams& p, int64_t old, int64_t add, int64_t held) {
    LaneNeed r;
    r.add = add > 0 ? add : 0;
    r.ok = old >= 0 && add >= 0 && held >= 0 && held <= p.max_pages &&
           old + add <= (int64_t)p.max_pages * p.page_size && held * p.page_size >= old;
    const int64_t want = ((old + add + p.page_size - 1) >> p.page_shift) - held;
    r.need = r.ok && want > 0 ? want : 0;
    return r;
}

// sums over the CTA before this thread (exclusive), and over all of it
__device__ void block_scan2(int64_t& a, int64_t& b, int64_t& sum_a, int64_t& sum_b, int64_t* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t xa = a, xb = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ya = __shfl_up_sync(~0u, xa, o), yb = __shfl_up_sync(~0u, xb, o);
        if (lane >= o) xa += ya, xb += yb;
    }
    if (lane == 31) sh[2 * warp] = xa, sh[2 * warp + 1] = xb;
    __syncthreads();
    int64_t pa = 0, pb = 0;
    sum_a = sum_b = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) pa = sum_a, pb = sum_b;
        sum_a += sh[2 * w], sum_b += sh[2 * w + 1];
    }
    a = pa + xa - a;
    b = pb + xb - b;
}

__global__ void __launch_bounds__(kThreads) gdn_page_plan_kernel(PagePlanParams p) {
    extern __shared__ int32_t smem[];
    __shared__ int64_t scan_sh[2 * kThreads / 32];
    __shared__ int last;
    int32_t* cu = smem;              // [B + 1] first token of each lane
    int32_t* from = smem + p.B + 1;  // [B] new pages of the lanes before it
    int32_t* kv = from + p.B;        // [B] cached tokens
    int32_t* held = kv + p.B;        // [B] pages
    int32_t* need = held + p.B;      // [B] new pages that it gets; -1: it gets none and its tokens no slots
    const int tid = threadIdx.x;
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    const int64_t taken0 = p.taken[0];
    const bool list_ok = taken0 >= 0 && taken0 <= p.num_pages;
    const int64_t base = list_ok ? taken0 : 0, left = list_ok ? p.num_pages - taken0 : 0;

    int64_t toks = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {  // the lengths are read once; new_lens waits in cu
        kv[b] = p.kv_lens[b];
        held[b] = p.held[b];
        cu[b] = p.new_lens[b];
        const LaneNeed n = lane_need(p, kv[b], cu[b], held[b]);
        toks += n.add;
        pages += n.need;
    }
    int64_t all_toks, all_pages;
    block_scan2(toks, pages, all_toks, all_pages, scan_sh);
    uint32_t bits = list_ok ? 0u : (uint32_t)GDN_ERRBIT_INDEX;
    if (all_toks > p.N) bits |= GDN_ERRBIT_SEQLEN;
    int64_t most = 0;  // pages that this thread's lanes bring the list to
    for (int b = b0; b < b1; ++b) {
        const int add = cu[b];
        const LaneNeed n = lane_need(p, kv[b], add, held[b]);
        const bool got = n.ok && (n.need == 0 || pages + n.need <= left);
        cu[b] = (int32_t)min(toks, (int64_t)INT32_MAX);
        from[b] = (int32_t)min(pages, (int64_t)INT32_MAX);
        need[b] = got ? (int32_t)n.need : -1;
        if (!n.ok) bits |= GDN_ERRBIT_SEQLEN;
        else if (!got) bits |= GDN_ERRBIT_PAGES;
        if (got && n.need > 0) most = pages + n.need;
        if (blockIdx.x == 0) p.total_lens[b] = got ? kv[b] + add : kv[b];
        toks += n.add;
        pages += n.need;
    }
    if (tid == 0) cu[p.B] = (int32_t)min(all_toks, (int64_t)INT32_MAX);
    __syncthreads();

    const int gsize = gridDim.x * kThreads, gtid = blockIdx.x * kThreads + tid;
    for (int b = gtid; b <= p.B; b += gsize) p.cu_seqlens[b] = cu[b];
    // the last lane that begins at x or before: lanes without tokens (or new pages) are passed over
    const int top = 1 << (31 - __clz(p.B));
    auto lane_of = [&](const int32_t* begin, int x) {
        int lo = 0;
        for (int s = top; s > 0; s >>= 1)
            if (lo + s < p.B && begin[lo + s] <= x) lo += s;
        return lo;
    };
    // new table entries
    const int fresh = (int)min(all_pages, left);
    for (int g = gtid; g < fresh; g += gsize) {
        const int b = lane_of(from, g);
        if (need[b] > 0) p.block_tables[(int64_t)b * p.max_pages + held[b] + g - from[b]] = p.free_pages[base + g];
    }
    // tokens, four of a thread side by side for the latency of their search and their pages
    const int64_t total = cu[p.B];
    for (int64_t t0 = gtid; t0 < p.N; t0 += 4 * (int64_t)gsize) {
        int pos[4], page[4];
        bool want[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t t = t0 + k * (int64_t)gsize;
            const int b = lane_of(cu, (int)min(t, (int64_t)INT32_MAX - 1)), col0 = held[b];
            pos[k] = t < total ? (int32_t)((uint32_t)kv[b] + (uint32_t)(t - cu[b])) : 0;
            want[k] = t < total && t < p.N && need[b] >= 0;
            const int col = pos[k] >> p.page_shift;
            page[k] = !want[k] ? -1 : col < col0 ? p.block_tables[(int64_t)b * p.max_pages + col] : p.free_pages[base + from[b] + col - col0];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t t = t0 + k * (int64_t)gsize;
            if (t >= p.N) break;
            const bool ok = page[k] >= 0 && page[k] < p.num_pages;
            if (want[k] && !ok) bits |= GDN_ERRBIT_INDEX;
            p.positions[t] = pos[k];
            p.slot_map[t] = ok ? (page[k] << p.page_shift) + (pos[k] & (p.page_size - 1)) : -1;
        }
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);

    __syncthreads();
    if (tid == 0) {
        last = 1;
        if (gridDim.x > 1) {
            __threadfence();
            last = atomicAdd(p.ticket, 1) == (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    // every CTA has read held and taken: they may be updated in place now
    for (int b = b0; b < b1; ++b) p.held_out[b] = held[b] + max(need[b], 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int64_t y = __shfl_xor_sync(~0u, most, o);
        most = y > most ? y : most;
    }
    if ((tid & 31) == 0) scan_sh[tid >> 5] = most;
    __syncthreads();
    if (tid == 0) {
        for (int w = 0; w < kThreads / 32; ++w) most = scan_sh[w] > most ? scan_sh[w] : most;
        p.taken_out[0] = (int32_t)(taken0 + most);
        if (gridDim.x > 1) *p.ticket = 0;
    }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanParams& p, cudaStream_t s) {
    // Shared memory is opened once on each device, for the most lanes: the default limit counts the kernel's static bytes too, and a
    // limit set by each call for its own lanes could be lowered by another thread before the launch.
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(gdn_page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kPlanMaxLanes));
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    // One CTA while that leaves its threads a few tokens and lanes each: it needs no ticket.  Then a CTA for 2048 tokens or
    // 128 lanes: more only repeat the scan.
    const int64_t want = ((int64_t)p.N + 2047) / 2048, lanes = (p.B + 127) / 128, most = want > lanes ? want : lanes;
    const int grid = p.N <= 4 * kThreads + 1024 && p.B <= kThreads ? 1 : (int)(most < 152 ? most : 152);
    gdn_page_plan_kernel<<<grid, kThreads, smem_bytes(p.B), s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
