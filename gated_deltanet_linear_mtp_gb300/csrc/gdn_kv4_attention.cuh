// gdn_kv4_attention.cuh -- what the two kernels of attention over the 4-bit cache share: a CTA's run of tiles, the warp that
// copies packed tiles by TMA, and the parts that several CTAs leave of one item.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_tcgen05.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// P = 2^(s - m) with the reference m = (running maximum) - kLift, which moves only where a score passes that maximum by more than
// kSlack (in units of log 2): P reaches 2^15, which f16 holds, and its subnormal steps of 2^-24 are 2^-31 of the row's largest or
// less.  With m at the maximum itself, keys below 2^-25 of the largest vanished from P V while they counted in l: with 16 keys
// above a million of them at e^-19, o lost all of its 3.5e-4.
constexpr float kSlack = 8.f;
constexpr float kLift = 7.f;

// A query row is held in f16 over the power of two of its largest number: the biased exponent, kept where the power and its
// reciprocal are normal numbers (NaN and infinity count as the largest), so a finite row loses nothing at either end of bf16.
__device__ __forceinline__ uint32_t row_exponent(uint32_t e) { return e < 1 ? 1 : e > 253 ? 253 : e; }
// What a score of such a row is multiplied by; finite, so that a score of 0 stays one
__device__ __forceinline__ float row_scale(const Kv4AttentionParams& p, uint32_t e, float scale) {
    const float x = __uint_as_float(e << 23) * scale * p.kv.k_scale * kLog2e;
    return fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
}

// Byte offset of 16-byte chunk c of token row r in a tile of codes, as TMA's swizzle of the row's size leaves it
template <int D>
__device__ __forceinline__ int code_off(int r, int c) {
    if (D == 64) return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
    if (D == 128) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * 128 + ((c ^ (r & 7)) << 4);
}

// A part's place in the workspace: O [rows][D], then m, l [rows]
__host__ __device__ constexpr int64_t part_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

// What a CTA left unfinished: the item that it began and the CTA that ends it
struct PartDesc {
    int32_t last;  // CTA that holds the item's last tile; -1: nothing to join
    int32_t rows;  // valid rows of the item
    int32_t q0;    // its first token's row in q
    int32_t r0;    // first row of the row tile
    int32_t hk;
    int32_t pad[3];
};

struct Lane {
    int q0, qlen, kv;  // first row in q, tokens (0: nothing to do), cached tokens
};

__device__ __forceinline__ Lane lane_extent(const Kv4AttentionParams& p, int b, uint32_t& bits) {
    int64_t a = (int64_t)b * p.T, n = p.T;
    if (p.cu_seqlens) {
        a = p.cu_seqlens[b];
        n = (int64_t)p.cu_seqlens[b + 1] - a;
    }
    Lane x{(int)a, (int)n, p.kv_lens[b]};
    if (a < 0 || n < 0 || n > p.T || a + n > p.N || x.kv < 0 || x.kv > (int64_t)p.max_pages * p.kv.page_size) {
        bits |= GDN_ERRBIT_SEQLEN;
        x.qlen = 0;
    }
    return x;
}

// The run of tiles of CTA c among `all`; the CTA that holds tile u
__device__ __forceinline__ int64_t run_begin(int64_t all, int64_t ctas, int64_t c) { return all * c / ctas; }
__device__ __forceinline__ int cta_of(int64_t all, int64_t ctas, int64_t u) {
    int64_t z = u * ctas / all;
    while (run_begin(all, ctas, z + 1) <= u) ++z;
    while (run_begin(all, ctas, z) > u) --z;
    return (int)z;
}

// One piece of a CTA's run: tiles kt0 .. kt1 - 1 of an item
struct Piece {
    int b, hk, r0, kt0, kt1, kts;
    Lane x;
};

template <typename C>
__device__ __forceinline__ int tiles_of(int kv) {
    return kv > 0 ? (kv - 1) / C::TILE + 1 : 1;
}

template <typename C>
__device__ __forceinline__ int64_t lane_tiles(const Kv4AttentionParams& p, const Lane& x) {
    return ((int64_t)x.qlen * p.G + C::ROWS - 1) / C::ROWS * (tiles_of<C>(x.kv) + C::SWITCH) * p.kv.HK;
}

// Walks a CTA's run of tiles u .. u1 - 1; lane `b` holds tile `base` first.  An item counts as C::SWITCH tiles more than it has,
// which are its first: a piece of these alone is passed over.
template <typename C>
struct Walk {
    int64_t u, u1, base;
    int b;
    __device__ __forceinline__ bool next(const Kv4AttentionParams& p, Piece& y) {
        uint32_t ignored = 0;
        while (u < u1) {
            y.x = lane_extent(p, b, ignored);
            int64_t n = lane_tiles<C>(p, y.x);
            while (base + n <= u) {
                base += n;
                y.x = lane_extent(p, ++b, ignored);
                n = lane_tiles<C>(p, y.x);
            }
            y.b = b;
            y.kts = tiles_of<C>(y.x.kv);
            const int64_t in = u - base, each = (int64_t)y.kts + C::SWITCH;
            const int item = (int)(in / each);
            const int64_t at = in - item * each, end = min(each, at + (u1 - u));
            y.hk = item % p.kv.HK;
            y.r0 = item / p.kv.HK * C::ROWS;
            y.kt0 = (int)max(at - C::SWITCH, (int64_t)0);
            y.kt1 = (int)max(end - C::SWITCH, (int64_t)0);
            u += end - at;
            if (y.kt1 > y.kt0) return true;
        }
        return false;
    }
};

// Sums of the lanes' tiles before each thread's lanes (`per` each) into s_scan [THREADS + 1]; all of the block's threads
template <typename C>
__device__ __forceinline__ void scan_lanes(const Kv4AttentionParams& p, int per, int64_t* s_scan, int64_t* s_warp, uint32_t& bits) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t x = 0;
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) x += lane_tiles<C>(p, lane_extent(p, b, bits));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += s_warp[w];
    s_scan[tid + 1] = x;
    if (tid == 0) s_scan[0] = 0;
    __syncthreads();
}

// The walk of this block's run
template <typename C>
__device__ __forceinline__ Walk<C> begin_walk(int per, const int64_t* s_scan, int64_t all, int64_t ctas) {
    Walk<C> walk;
    walk.u = run_begin(all, ctas, blockIdx.x);
    walk.u1 = run_begin(all, ctas, (int64_t)blockIdx.x + 1);
    int lo = 0, hi = C::THREADS;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_scan[mid] <= walk.u) lo = mid;
        else hi = mid;
    }
    walk.b = lo * per;
    walk.base = s_scan[lo];
    return walk;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// The copying warp: tiles of the run, page by page; lane i takes page i of a tile.  A stage holds a tile's keys and values
// (codes of both, then scales of both), or with C::SPLIT its keys or its values, which are then a warp's each (kind 0, 1):
// with pages of 16 tokens one warp's 16 copies a stage are too slow for the prompts' kernel.
template <typename C, typename W>
__device__ __forceinline__ void produce(const Kv4AttentionParams& p, const CUtensorMap* map, W walk, uint32_t pool,
                                        uint8_t* pool_p, uint32_t full, uint32_t empty, uint32_t& bits, int kind = 0) {
    constexpr int KINDS = C::SPLIT ? 1 : 2;  // of rows in a stage
    const int lane = threadIdx.x & 31, P = p.kv.page_size, HK = p.kv.HK;
    const int PR = P < C::TILE ? P : C::TILE;  // rows of a copy
    uint32_t it = 0;
    bool late = false;
    Piece y;
    while (!late && walk.next(p, y)) {
        const int32_t* table = p.block_tables + (int64_t)y.b * p.max_pages;
        auto entry = [&](int kt) {  // this lane's page of tile kt
            const int tok = kt * C::TILE + lane * PR;
            return kt < y.kt1 && lane * PR < C::TILE && tok < y.x.kv ? table[tok / P] : -2;
        };
        int pg = entry(y.kt0);
        for (int kt = y.kt0; kt < y.kt1 && !late; ++kt) {
            const int ahead = entry(kt + 1);
            for (int part = 0; part < 2 / KINDS; ++part, ++it) {
                if (C::SPLIT && part != kind) continue;
                const uint32_t s = it % C::STAGES, round = it / C::STAGES;
                if (round > 0 && !__all_sync(~0u, mbar_wait_bounded(empty + 8 * s, (round - 1) & 1, GDN_WAIT_POLLS))) {
                    bits |= GDN_ERRBIT_TIMEOUT;
                    late = true;
                    break;
                }
                const uint32_t st = pool + s * C::STAGE, bar = full + 8 * s;
                const bool here = pg != -2, ok = here && (uint32_t)pg < (uint32_t)p.kv.num_pages;
                if (here && !ok) {  // a page outside the cache: zeros
                    bits |= GDN_ERRBIT_INDEX;
                    uint8_t* z = pool_p + s * C::STAGE;
                    for (int i = 0; i < KINDS; ++i) {
                        for (int j = 0; j < PR * C::CB; j += 16)
                            *reinterpret_cast<uint4*>(z + (i * C::TILE + lane * PR) * C::CB + j) = make_uint4(0, 0, 0, 0);
                        for (int j = 0; j < PR * C::SB; j += 16)
                            *reinterpret_cast<uint4*>(z + KINDS * C::TILE * C::CB + (i * C::TILE + lane * PR) * C::SB + j) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                const uint32_t n = __popc(__ballot_sync(~0u, ok));
                __syncwarp();  // the lanes' zeros come before the arrival that tells of them (a vote orders no memory)
                if (lane == 0) mbar_arrive_expect_tx(bar, n * (uint32_t)(KINDS * PR * (C::CB + C::SB)));
                __syncwarp();
                if (ok) {
                    const int off = (kt * C::TILE) & (P - 1);
#pragma unroll
                    for (int i = 0; i < KINDS; ++i) {
                        const int which = part + i;
#ifdef GDN_TEST_MISSING_COPY
                        if (y.b == 0 && y.hk == 0 && y.r0 == 0 && kt == 0 && which == 0 && lane == 0) continue;
#endif
                        tma_load_4d(st + (i * C::TILE + lane * PR) * C::CB, map, 0, off, which * HK + y.hk, pg, bar);
                        const int64_t row = (((int64_t)pg * 2 + which) * HK + y.hk) * P + off;
                        bulk_g2s(st + KINDS * C::TILE * C::CB + (i * C::TILE + lane * PR) * C::SB, p.kv.scales + row * C::SB,
                                 (uint32_t)(PR * C::SB), bar);
                    }
                }
            }
            pg = ahead;
        }
    }
    // no copy outlives the CTA
    for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; i < it; ++i)
        mbar_wait_bounded(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, GDN_WAIT_POLLS);
}

// ---- tensor memory ----------------------------------------------------------------------------------------------
// instruction descriptor of tcgen05.mma kind::f16 with f16 operands, D fp32
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The wait for this thread's loads, and that what they loaded is not used before it
__device__ __forceinline__ void tmem_wait_ld16(float (&f)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]), "+f"(f[8]),
                   "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15])
                 :
                 : "memory");
}

// ---- host ---------------------------------------------------------------------------------------------------
// The codes as TMA sees them: [num_pages][2 HK][page_size][D / 2 bytes], copied by page (a tile at most)
inline cudaError_t codes_map(const Kv4& kv, int tile, CUtensorMap* map) {
    const EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t CB = (cuuint64_t)kv.D / 2, P = (cuuint64_t)kv.page_size;
    const cuuint64_t dims[4] = {CB, P, (cuuint64_t)2 * kv.HK, (cuuint64_t)kv.num_pages};
    const cuuint64_t strides[3] = {CB, CB * P, CB * P * 2 * kv.HK};
    const cuuint32_t box[4] = {(cuuint32_t)CB, (cuuint32_t)(P < (cuuint64_t)tile ? P : (cuuint64_t)tile), 1, 1}, one[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle sw = kv.D == 64    ? CU_TENSOR_MAP_SWIZZLE_32B
                                  : kv.D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, kv.codes, dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The second kernel of a call: joins the parts that `ctas` CTAs left of items of up to `rows` rows (gdn_kv4_attention.cu)
cudaError_t launch_kv4_join(const Kv4AttentionParams& p, int rows, int ctas, cudaStream_t s);
// The kernel for many rows (gdn_kv4_attention_wide.cu)
cudaError_t launch_kv4_attention_wide(const Kv4AttentionParams& p, cudaStream_t s);
int64_t kv4_attention_wide_workspace(int D);

}  // namespace gdn
