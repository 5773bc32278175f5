// gdn_kv4_attention_wide.cu -- attention over the 4-bit cache for lanes of many rows (prompts): the same operation as
// gdn_kv4_attention.cu, on the tensor cores of tcgen05.
//
// Bound: the products, 4 D flops a row and key.  An item is a tile of MT * 128 rows (whole tokens times the G heads of a key
// head) of one lane and key head; a CTA takes its tiles of TILE keys in turn, as four kinds of warps:
//   * two warps copy the packed tiles into shared memory by TMA, keys and values (shared with the decode kernel);
//   * a warpgroup unpacks them into f16 operand tiles (128-byte swizzle, a ring of two pairs), once for all rows: a
//     number costs the unpacking 1/256 of its products;
//   * a thread for each 128 rows issues the MMAs: S = Q K^T into tensor memory, O += P V with P read from tensor memory;
//   * a warpgroup for each 128 rows takes a row of S a thread, forms P in place of S as f16 and keeps the row's statistics.
// S goes by units of 64 keys in two buffers: the way from a product to its softmax and back takes longer than either
// (about 600 cycles each way), and with one buffer of 128 keys the tensor cores waited for it (665 us for two chunks of 2048
// tokens behind 8192 keys, HQ 32, HK 4, D 128, against 573 then).  An item of up to 128 rows is worked on by both halves of the
// CTA, each with half of every tile's keys (256 lanes of 64 rows over up to 4096 keys, D 64: 229 us against 255 then).
// Measured (graph replays): those two chunks 531 us, 1.17 PFLOP/s; 16 ragged prompts of up to 2048 tokens, HQ 16, HK 2, D 128, 136 us,
// 0.54 PFLOP/s; the 256 lanes 160 us, 0.98 TB/s.  At other head dimensions: the two chunks at D 64 488 us, and with HQ 16, HK 2, D 256
// 873 us; the ragged prompts at D 64 113 us, at D 256 333 us.  What is left above the products is waiting: a unit of 64 keys takes 2000
// cycles where its products take 1280 (128 rows each), since a warp's softmax is one chain of loads, maxima, exponentials and stores
// with two warps a scheduler to cover it; and an item's begin and end.
// The reference m of P = 2^(s - m) moves only where a score passes the running maximum by more than 8 (in units of log 2; then
// that thread scales its row of O in tensor memory), so O stays in tensor memory throughout.
// Queries, P and statistics are held as in the decode kernel: f16 by a power of two a row, f16 lifted by kLift, fp32.
//
// Work split: all tiles of all items are numbered and each CTA (one an SM) takes an equal run of them, since the rows of a
// prompt see anything from few to all keys and items of whole rows leave SMs idle at the end; parts are joined by the decode
// kernel's second launch.
#include <atomic>

#include "gdn_kv4_attention.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 512;  // 4 warpgroups: softmax, softmax or unpacking, unpacking, MMA and copies
constexpr int kMmaWarp = 12, kLoadWarp = 14;  // kMmaWarp + m issues the products of rows 128 m ..; two warps copy
// Tiles that the begin and the end of an item count as in the split of the work (a piece of n tiles takes about 4.2 n + 10.7
// thousand cycles at D 128).  16 ragged prompts of up to 2048 tokens, HQ 16, HK 2, in us with 0 to 5: D 128 220, 171, 146, 135, 135,
// 139; D 64 162, 127, 109, 114, 115, 119; D 256 489, 412, 380, 333, 314, 322.  Chunks of 2048 behind 8192 keys differ by 2 % at most.
constexpr int kSwitch = 3;
constexpr int kLaunchRegs = 128, kSoftRegs = 160, kUnpackRegs = 112, kRestRegs = 80;
static_assert(2 * kSoftRegs + kUnpackRegs + kRestRegs <= 4 * kLaunchRegs, "the block's registers");

template <int D_>
struct Wide {
    static constexpr int D = D_;
    static constexpr int MT = D == 256 ? 1 : 2;        // tiles of 128 rows
    static constexpr int TILE = D == 256 ? 64 : 128;   // keys of a tile
    static constexpr int ROWS = MT * 128;
    static constexpr bool SPLIT = true;                // a stage of the copies holds keys or values
    static constexpr int PAIRS = D == 64 ? 4 : 2;      // places of the ring of unpacked tiles: V of one tile, K of the next
    static constexpr int STAGES = D == 64 ? 6 : 3;
    static constexpr int CB = D / 2, SB = D / 16, STAGE = TILE * (CB + SB);
    static constexpr int UNPACK = 128 * (3 - MT);      // threads that unpack
    static constexpr int QBYTES = 128 * D * 2, KVBYTES = TILE * D * 2;
    static constexpr int Q_AT = 0, RING_AT = MT * QBYTES, POOL_AT = RING_AT + 2 * PAIRS * KVBYTES;
    static constexpr int SMEM = 1024 + POOL_AT + STAGES * STAGE;
    static constexpr int UNIT = 64, UPT = TILE / UNIT;  // keys of a product S; of them in a tile
    static constexpr int O_COL = 0, S_COL = MT * D, COLS = 512;
    static_assert(S_COL + MT * 2 * UNIT <= COLS, "tensor memory");
};

// The thread's row of `cols` columns (a multiple of 8) times f: fp32, or two f16 a column
template <bool HALF>
__device__ __noinline__ void scale_columns(uint32_t col, int cols, float f) {
    tmem_wait_st();
    for (int c = 0; c < cols; c += 8) {
        float v[16];
        uint32_t w[8];
        tmem_ld16(col + c, v);  // of which the first 8 are used
        tmem_wait_ld16(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (HALF) {
                const uint32_t b = __float_as_uint(v[j]);
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&b));
                w[j] = f16x2_bits(x.x * f, x.y * f);
            } else {
                w[j] = __float_as_uint(v[j] * f);
            }
        }
        tmem_st8(col + c, w);
    }
    tmem_wait_st();
}

// ---- the run of tiles: pairs (lane, row tile), each with a tile of keys for every key head ------------------------
// tt: tokens of a row tile
__device__ __forceinline__ int row_tiles(const Lane& x, int tt) { return (x.qlen + tt - 1) / tt; }

// Tiles of keys that row tile rt of a lane sees
template <typename C>
__device__ __forceinline__ int key_tiles(const Lane& x, int tt, int rt) {
    const int keys = x.kv - x.qlen + min((rt + 1) * tt, x.qlen);  // qlen <= N, kv: both below 2^31
    return keys > 0 ? (keys - 1) / C::TILE + 1 : 1;
}

template <typename C>
struct WideWalk {
    int64_t u, u1, base;  // base: first tile of pair (b, rt)
    int b, rt, tt;
    Lane x;  // of lane b
    __device__ __forceinline__ bool next(const Kv4AttentionParams& p, Piece& y) {
        if (u >= u1) return false;
        uint32_t ignored = 0;
        for (;;) {
            if (rt * tt >= x.qlen) {
                rt = 0;
                x = lane_extent(p, ++b, ignored);
                continue;
            }
            y.kts = key_tiles<C>(x, tt, rt);
            const int64_t pair = (int64_t)(y.kts + kSwitch) * p.kv.HK;
            if (base + pair <= u) {
                base += pair;
                ++rt;
                continue;
            }
            const uint32_t in = (uint32_t)(u - base), each = (uint32_t)y.kts + kSwitch;  // in is below each * HK
            y.hk = (int)(in / each);
            const int at = (int)(in - (uint32_t)y.hk * each), end = (int)min((int64_t)each, at + (u1 - u));
            u += end - at;
            y.kt0 = max(at - kSwitch, 0);
            y.kt1 = max(end - kSwitch, 0);
            if (y.kt1 > y.kt0) break;
            if (u >= u1) return false;
        }
        y.x = x;
        y.b = b;
        y.r0 = rt * tt * p.G;
        return true;
    }
};

// Sum over the threads before this one, and over all, of a number each
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* s_warp, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t z = __shfl_up_sync(~0u, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = y;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    return before + y - x;
}

// The lane and row tile of pair i; s_pairs[t]: pairs before the lanes of thread t (`per` lanes each)
__device__ __forceinline__ void locate(const Kv4AttentionParams& p, const int64_t* s_pairs, int per, int tt, int64_t i, int& b, int& rt) {
    int lo = 0, hi = kThreads;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pairs[mid] <= i) lo = mid;
        else hi = mid;
    }
    uint32_t ignored = 0;
    int64_t at = s_pairs[lo];
    b = lo * per;
    for (;;) {
        const int n = row_tiles(lane_extent(p, b, ignored), tt);
        if (at + n > i) break;
        at += n;
        ++b;
    }
    rt = (int)(i - at);
}

// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// An item of up to 128 rows: both warpgroups of the softmax and both issuing threads take all of its rows, each with half of
// every tile's keys (a lane's last item alone has so few: 256 / G * G is above 192 for G <= 64)
template <typename C>
__device__ __forceinline__ bool in_halves(const Kv4AttentionParams& p, const Piece& y) {
    return C::MT == 2 && y.x.qlen * p.G - y.r0 <= 128;
}

template <typename C>
__global__ void __launch_bounds__(kThreads, 1) gdn_kv4_attention_wide_kernel(const __grid_constant__ Kv4AttentionParams p,
                                                                             const __grid_constant__ CUtensorMap map) {
    constexpr int D = C::D, MT = C::MT, TILE = C::TILE;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t s_warp[kThreads / 32];
    __shared__ uint64_t s_bar[2 * C::STAGES + 2 * C::PAIRS + 8 * MT + 2];
    __shared__ float2 s_ml[MT * 128];  // the two warpgroups' statistics of rows that they share
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t base_u = smem_u32(smem);
    int64_t* s_pairs = reinterpret_cast<int64_t*>(smem + C::RING_AT);  // [kThreads + 1], before the ring is filled
    int64_t* s_tiles = s_pairs + kThreads + 1;                         // [kThreads + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw_full = smem_u32(s_bar), raw_empty = raw_full + 8 * C::STAGES, kv_full = raw_empty + 8 * C::STAGES,
                   kv_empty = kv_full + 8 * C::PAIRS, q_full = kv_empty + 8 * C::PAIRS, s_full = q_full + 8 * MT,
                   p_full = s_full + 16 * MT, pv_prev = p_full + 16 * MT, pv_last = pv_prev + 8 * MT,
                   idle = pv_last + 8 * MT, told = idle + 8 * MT, read = told + 8;
    // s_full, p_full: two for each 128 rows; pv_prev, pv_last: the last P V of a piece but one, and the last; idle: all
    // products are done; told, read: both warpgroups' halves of shared rows are complete, and have been read
    uint32_t bits = 0;

    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) mbar_init(raw_full + 8 * i, 1), mbar_init(raw_empty + 8 * i, C::UNPACK / 32);
        for (int i = 0; i < C::PAIRS; ++i) mbar_init(kv_full + 8 * i, C::UNPACK / 32), mbar_init(kv_empty + 8 * i, MT);
        for (int i = 0; i < MT; ++i) mbar_init(q_full + 8 * i, 4), mbar_init(pv_prev + 8 * i, 1), mbar_init(pv_last + 8 * i, 1), mbar_init(idle + 8 * i, 1);
        for (int i = 0; i < 2 * MT; ++i) mbar_init(s_full + 8 * i, 1), mbar_init(p_full + 8 * i, 4);
        mbar_init(told, 8), mbar_init(read, 8);
        fence_mbar_init();
        s_dead = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), C::COLS);

    // ---- this CTA's run of tiles --------------------------------------------------------------------------
    WideWalk<C> walk;
    int64_t all;
    {
        const int per = (p.B + kThreads - 1) / kThreads, tt = C::ROWS / p.G;
        int64_t n = 0, pairs;
        for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) n += row_tiles(lane_extent(p, b, bits), tt);
        s_pairs[tid] = block_scan(n, s_warp, pairs);
        if (tid == 0) s_pairs[kThreads] = pairs;
        __syncthreads();
        const int64_t i0 = pairs * tid / kThreads, i1 = pairs * (tid + 1) / kThreads;
        n = 0;
        if (i0 < i1) {
            int b, rt;
            uint32_t ignored = 0;
            locate(p, s_pairs, per, tt, i0, b, rt);
            Lane x = lane_extent(p, b, ignored);
            for (int64_t i = i0; i < i1; ++i, ++rt) {
                while (rt * tt >= x.qlen) {
                    rt = 0;
                    x = lane_extent(p, ++b, ignored);
                }
                n += key_tiles<C>(x, tt, rt) + kSwitch;
            }
        }
        s_tiles[tid] = block_scan(n * p.kv.HK, s_warp, all);
        if (tid == 0) s_tiles[kThreads] = all;
        __syncthreads();
        const int64_t ctas = all < gridDim.x ? all : gridDim.x;
        walk.u = walk.u1 = 0;
        if (blockIdx.x < ctas) {
            walk.u = run_begin(all, ctas, blockIdx.x);
            walk.u1 = run_begin(all, ctas, (int64_t)blockIdx.x + 1);
            int lo = 0, hi = kThreads;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_tiles[mid] <= walk.u) lo = mid;
                else hi = mid;
            }
            walk.base = s_tiles[lo];
            uint32_t ignored = 0;
            locate(p, s_pairs, per, tt, pairs * lo / kThreads, walk.b, walk.rt);
            walk.x = lane_extent(p, walk.b, ignored);
            walk.tt = tt;
        }
    }
    const int64_t ctas = all < gridDim.x ? all : gridDim.x;
    PartDesc* desc = reinterpret_cast<PartDesc*>(p.workspace) + blockIdx.x;
    float* parts = reinterpret_cast<float*>(reinterpret_cast<PartDesc*>(p.workspace) + gridDim.x);
    if (tid == 0) desc->last = -1;
    if (bits && p.err && blockIdx.x == 0) atomicOr(p.err, (int32_t)bits);
    bits = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* dead = &s_dead;
    auto wait = [&](uint32_t bar, uint32_t parity) {  // false: it ran out, and the CTA's work with it
        for (uint32_t i = 0; i < GDN_WAIT_POLLS; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((i & 63) == 63 && *dead) return false;
        }
        *dead = 1;
        bits |= GDN_ERRBIT_TIMEOUT;
        return false;
    };
    auto warp_wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(~0u, wait(bar, parity)) != 0; };

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
        if (warp >= kLoadWarp) {
            produce<C>(p, &map, walk, base_u + C::POOL_AT, smem + C::POOL_AT, raw_full, raw_empty, bits, warp - kLoadWarp);
        } else if (warp < kMmaWarp + MT && lane == 0) {
            // The ring holds pairs: pair j of a piece is V of its tile j - 1 and K of its tile j (the first has K alone, the
            // last V alone), since a unit's P V and the scores two units on need them together.  A thread for each 128 rows:
            // what one waits for (250 cycles even for what is ready, as it queues behind the products) passes while the
            // other's products run.  Units of 64 keys alternate between two buffers of S, so that a softmax finds its next
            // scores ready whatever the way there and back takes.
            constexpr uint32_t id_s = idesc_f16(128, C::UNIT), id_o = idesc_f16(128, D) | (1u << 16);
            const int m = warp - kMmaWarp;
            uint32_t pair = 0, piece = 0, unit = 0;  // ring pairs before this piece; pieces and units of these rows
            Piece y;
            bool go = true;
            auto pair_wait = [&](uint32_t n) { return wait(kv_full + 8 * (n % C::PAIRS), (n / C::PAIRS) & 1); };
            // descriptors differ in their start address alone: 16 bytes count 1
            const uint64_t q_desc = umma_desc_sw128(base_u + C::Q_AT + m * C::QBYTES),
                           k_desc = umma_desc_sw128(base_u + C::RING_AT + C::KVBYTES),
                           v_desc = umma_desc_sw128_mn(base_u + C::RING_AT, TILE * 128);
            int upt = C::UPT;  // units of a tile that these rows take
            bool halves = false;
            auto sub = [&](int u) { return halves ? m : u % C::UPT; };  // which of its tile's units unit u is
            auto product_s = [&](int u) {  // scores of unit u of the piece
                const uint32_t n = pair + u / upt, at = unit + u;
                const uint64_t k = k_desc + (n % C::PAIRS) * (2 * C::KVBYTES / 16) + sub(u) * (C::UNIT * 128 / 16);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma_bf16(tmem + C::S_COL + (2 * m + (at & 1)) * C::UNIT, q_desc + ((ks / 4) * 128 * 128 + (ks % 4) * 32) / 16,
                              k + ((ks / 4) * TILE * 128 + (ks % 4) * 32) / 16, id_s, ks > 0);
                umma_commit(s_full + 8 * (2 * m + (at & 1)));
            };
            while (go && walk.next(p, y)) {
                halves = in_halves<C>(p, y);
                upt = halves ? 1 : C::UPT;
                const int n = y.kt1 - y.kt0, units = n * upt;
                int have = 0;  // pairs of the piece that are known to be there
                auto need = [&](int q) {
                    for (; go && have <= q; ++have) go = pair_wait(pair + have);
                };
                for (int u = 0; u < 2 && u < units && go; ++u) {
                    need(u / upt);
                    if (u == 0) go = go && wait(q_full + 8 * m, piece & 1);
                    if (!go) break;
                    tc_fence_after();
                    product_s(u);
                    if (u == upt - 1) umma_commit(kv_empty + 8 * (pair % C::PAIRS));
                }
                auto need_for = [&](int u) {  // P V of unit u, and the scores of unit u + 1
                    if (u < units) need(u / upt + 1);
                };
                need_for(0);
                for (int u = 0; u < units && go; ++u) {
                    const uint32_t at = unit + u, nv = pair + u / upt + 1;
                    go = wait(p_full + 8 * (2 * m + (at & 1)), (at >> 1) & 1);
                    if (!go) break;
                    tc_fence_after();
                    const uint64_t v = v_desc + (nv % C::PAIRS) * (2 * C::KVBYTES / 16) + sub(u) * (C::UNIT * 128 / 16);
#pragma unroll
                    for (int ks = 0; ks < C::UNIT / 16; ++ks)
                        umma_bf16_ta(tmem + C::O_COL + m * D, tmem + C::S_COL + (2 * m + (at & 1)) * C::UNIT + ks * 8,
                                     v + ks * (2048 / 16), id_o, u > 0 || ks > 0);
                    need_for(u + 1);  // while P V runs; then P is all that the next unit waits for (no pair further on: its
                                      // place in the ring is freed by the commit below)
                    if (!go) break;
                    if (u + 2 < units) product_s(u + 2);
                    else umma_commit((u + 1 < units ? pv_prev : pv_last) + 8 * m);  // scores two units on tell of the others
                    if (u % upt == upt - 1) umma_commit(kv_empty + 8 * (nv % C::PAIRS));
                }
                ++piece;
                unit += units;
                pair += n + 1;
            }
            umma_commit(idle + 8 * m);  // no product outlives the CTA's memory, whatever wait ran out
            if (!mbar_wait_bounded(idle + 8 * m, 0, GDN_WAIT_POLLS)) bits |= GDN_ERRBIT_TIMEOUT;
        }
    } else if (warp >= 4 * MT) {
        // ---- unpacking: thread (row, part of its dimensions) -------------------------------------------------
        if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kUnpackRegs));
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        constexpr int PARTS = C::UNPACK / TILE, RUN = D / PARTS;  // dimensions of a thread
        const int idx = tid - 128 * MT, r = idx % TILE, part = idx / TILE;
        uint32_t pair = 0, stage = 0;  // ring pairs; stages of the copies
        Piece y{};
        bool go = true;
        auto tile = [&](int kt, bool values, uint8_t* dst) {  // the next stage into an operand tile
            const uint32_t st = stage % C::STAGES;
            go = warp_wait(raw_full + 8 * st, (stage / C::STAGES) & 1);
            if (!go) return;
            ++stage;
            const bool real = kt * TILE + r < y.x.kv;  // what lies behind the last token may be anything
            const uint8_t* codes = smem + C::POOL_AT + st * C::STAGE;
            const uint8_t* sc = codes + TILE * C::CB + r * C::SB + part * (RUN / 16);
            uint4 w[RUN / 32];
            uint32_t two[RUN / 32];
#pragma unroll
            for (int c = 0; c < RUN / 32; ++c) {  // 16 bytes of codes: 32 dimensions, two scales
                w[c] = *reinterpret_cast<const uint4*>(codes + code_off<D>(r, part * (RUN / 32) + c));
                two[c] = real ? *reinterpret_cast<const uint16_t*>(sc + 2 * c) : 0u;
            }
#pragma unroll
            for (int c = 0; c < RUN / 32; ++c) {
                uint32_t f2 = e4m3x2_to_f16(two[c]);
                if (values) f2 = nan_as_zero(f2);  // a token that does not see the value has 0 for P
                const uint32_t sf[2] = {__byte_perm(f2, f2, 0x1010), __byte_perm(f2, f2, 0x3232)};
                const uint32_t ws[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t f[4];
                    e2m1x8_to_f16(ws[j], f);
#pragma unroll
                    for (int x = 0; x < 4; ++x) f[x] = hmul2(f[x], sf[j >> 1]);
                    *reinterpret_cast<uint4*>(dst + sw128(TILE, r, (part * (RUN / 32) + c) * 4 + j)) = make_uint4(f[0], f[1], f[2], f[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_empty + 8 * st);
        };
        while (go && walk.next(p, y)) {
            for (int kt = y.kt0; kt <= y.kt1 && go; ++kt, ++pair) {  // V of tile kt - 1, K of tile kt
                const uint32_t at = pair % C::PAIRS;
                if (pair >= C::PAIRS) go = warp_wait(kv_empty + 8 * at, (pair / C::PAIRS - 1) & 1);
                uint8_t* dst = smem + C::RING_AT + at * 2 * C::KVBYTES;
#pragma unroll 1
                for (int which = kt > y.kt0 ? 0 : 1; which < (kt < y.kt1 ? 2 : 1) && go; ++which)
                    tile(kt - 1 + which, which == 0, dst + which * C::KVBYTES);
                if (!go) break;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(kv_full + 8 * at);
            }
        }
    } else {
        // ---- softmax: one row a thread ---------------------------------------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int mt = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // lane 32 (warp mod 4) in the upper half
        const uint32_t s_col0 = lanes + C::S_COL + mt * 2 * C::UNIT, o_col = lanes + C::O_COL + mt * D;
        const uint32_t magic = 65535u / (uint32_t)p.G + 1u;  // x / G = x * magic >> 16 for x < 256 and G <= 64
        uint32_t unit = 0, piece = 0, prev = 0;  // of this warpgroup: units, pieces, and pieces of more than one unit
        uint32_t shared = 0;                     // pieces in halves
        Piece y;
        bool go = true;
        while (go && walk.next(p, y)) {
            const bool halves = in_halves<C>(p, y);
            const int row0 = halves ? 0 : mt * 128;  // the warpgroup's first row of the item
            // an item's rows are those of its whole tokens: where G does not divide the tile, the places behind them stay empty
            // (what follows is the next item's, whose keys go further)
            const int n = y.kt1 - y.kt0, units = halves ? n : n * C::UPT, nrows = min(walk.tt * p.G, y.x.qlen * p.G - y.r0), r = row0 + row;
            const bool mine = r < nrows;
            // rows of q and o lie at `first` + the row's `rel` rows; a row of 128 is loaded by LR lanes, 16 bytes each
            constexpr int LR = D / 8, RPI = 32 / LR;
            const int wrow = (warp & 3) * 32;  // the warp's first row of its 128
            uint8_t* stage = smem + C::Q_AT + mt * C::QBYTES;
            const int t_first = y.r0 / p.G;
            const int64_t first_row = (int64_t)(y.x.q0 + t_first) * p.HQ + y.hk * p.G;
            const int rt = (int)((uint32_t)r * magic >> 16), rel = mine ? rt * p.HQ + r - rt * p.G : 0;
            // Q: the rows as they are, then each thread its own as f16, scaled by a power of two (and by the sign of p.scale).
            // Short loops: a piece's start is cold code for the instruction cache (with the rows' maxima by shuffles
            // and eight rows unrolled, 16 ragged prompts took 234 us).
#pragma unroll 4
            for (int i = 0; i < LR; ++i) {
                const int at = i * RPI + lane / LR, lr = wrow + at;
                const int64_t off = (first_row + __shfl_sync(~0u, rel, at)) * D + (lane % LR) * 8;
                cp_async16(smem_u32(stage + sw128(128, lr, lane % LR)), (const __nv_bfloat16*)p.q + off, row0 + lr < nrows);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            uint32_t top2 = 0;  // of each half of a word: magnitudes order as integers
#pragma unroll 4
            for (int c = 0; c < LR; ++c) {
                const uint4 w = *reinterpret_cast<const uint4*>(stage + sw128(128, row, c));
                top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
            }
            const uint32_t e = row_exponent(max(top2 & 0xffffu, top2 >> 16) >> 7);
            const float down = __uint_as_float((254u - e) << 23) * (p.scale < 0.f ? -1.f : 1.f);
            // (at least 2^-120: a masked score of -inf must stay one)
            const float sc = fmaxf(row_scale(p, e, fabsf(p.scale)), 0x1p-120f);
#pragma unroll 2
            for (int c = 0; c < LR; ++c) {
                uint4* at = reinterpret_cast<uint4*>(stage + sw128(128, row, c));
                const uint4 w = *at;
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                uint32_t f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = bf16x2_to_float2(ws[j]);
                    f[j] = f16x2_bits(v.x * down, v.y * down);
                }
                *at = make_uint4(f[0], f[1], f[2], f[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + 8 * mt);
            const int t = t_first + rt;
            const int limit = y.x.kv - y.x.qlen + t + 1;                   // keys that the row sees
            const int all_see = y.x.kv - y.x.qlen + y.r0 / p.G + 1;        // that every row of the item sees
            float m = -INFINITY, l = 0.f;
            for (int u = 0; u < units && go; ++u, ++unit) {
                go = warp_wait(s_full + 8 * (2 * mt + (unit & 1)), (unit >> 1) & 1);
                if (!go) break;
                tc_fence_after();
                const uint32_t s_col = s_col0 + (unit & 1) * C::UNIT;
                const int first = halves ? (y.kt0 + u) * TILE + mt * C::UNIT : y.kt0 * TILE + u * C::UNIT;
                const bool mask = first + C::UNIT > all_see;
                F2 l2 = f2(0.f, 0.f);
                // 16 columns at a time, P's 8 where S has been read, and not unrolled: the loop's instructions stay in the
                // scheduler's cache, which four kinds of warps share (unrolled over all 64 columns 595 us against 540 then)
#pragma unroll 1
                for (int c = 0; c < C::UNIT; c += 16) {
                    float x[16];
                    tmem_ld16(s_col + c, x);
                    tmem_wait_ld16(x);
                    if (mask) {
                        const int lim = limit - first - c;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j >= lim) x[j] = -INFINITY;
                    }
                    float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int j = 4; j < 16; ++j) t4[j & 3] = fmaxf(t4[j & 3], x[j]);
                    const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sc;
                    const bool move = top > m + (kSlack + kLift);
                    if (__any_sync(~0u, move)) {
                        const float mn = move ? top - kLift : m;
                        const float f = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
                        m = mn;
                        l *= f;
                        l2 = mul(l2, f2(f, f));
                        if (u > 0) {  // the product that last wrote O came before the next unit's scores, or is the last but one
                            go = u + 1 < units ? warp_wait(s_full + 8 * (2 * mt + ((unit + 1) & 1)), ((unit + 1) >> 1) & 1)
                                               : warp_wait(pv_prev + 8 * mt, prev & 1);
                            tc_fence_after();
                            scale_columns<false>(o_col, D, f);
                        }
                        scale_columns<true>(s_col, c / 2, f);
                    }
                    const float mm = m == -INFINITY ? 0.f : -m;
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 z = split(fma(f2(x[2 * j], x[2 * j + 1]), f2(sc, sc), f2(mm, mm)));
                        const float a = exp2_fast(z.x), b = exp2_fast(z.y);
                        l2 = add(l2, f2(a, b));
                        w[j] = f16x2_bits(a, b);
                    }
                    tmem_st8(s_col + c / 2, w);
                }
                const float2 ls = split(l2);
                l += ls.x + ls.y;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * (2 * mt + (unit & 1)));
            }
            go = go && warp_wait(pv_last + 8 * mt, piece & 1);
            if (!go) break;
            ++piece;
            prev += units > 1;
            tc_fence_after();
            // rows in halves: the statistics joined; each warpgroup then puts out half of the dimensions
            float fa = 1.f, fb = 1.f;  // factors of the first and the second warpgroup's O
            if (halves) {
                s_ml[mt * 128 + row] = make_float2(m, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(told);
                go = warp_wait(told, shared & 1);
                if (!go) break;
                tc_fence_after();
                const float2 a = s_ml[row], b = s_ml[(MT - 1) * 128 + row];
                m = fmaxf(a.x, b.x);
                fa = m == -INFINITY ? 1.f : exp2_fast(a.x - m);
                fb = m == -INFINITY ? 1.f : exp2_fast(b.x - m);
                l = fmaf(a.y, fa, b.y * fb);
            }
            const bool whole = y.kt0 == 0 && y.kt1 == y.kts;
            float* part = parts + ((int64_t)blockIdx.x * 2 + (y.kt0 == 0 ? 1 : 0)) * part_floats(C::ROWS, D);
            const float inv = l > 0.f ? p.kv.v_scale / l : l != l ? l : 0.f;
            // rows go out through Q's place in shared memory, so that a row's lanes store side by side; in Q's layout, since then a
            // warp's rows are its own and another warp may be at the next piece's Q already
            auto put_out = [&](int col0, int cols) {  // dimensions col0 ..; a row's place holds D bf16 or D / 2 fp32
#pragma unroll 1
                for (int c = 0; c < cols; c += 16) {
                    float v[16];
                    if (halves) {
                        float v2[16];
                        const uint32_t o_first = lanes + C::O_COL + col0 + c;
                        tmem_ld16(o_first, v);
                        tmem_ld16(o_first + (MT - 1) * D, v2);
                        tmem_wait_ld16(v);
                        tmem_wait_ld16(v2);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = fmaf(v[j], fa, v2[j] * fb);
                    } else {
                        tmem_ld16(o_col + col0 + c, v);
                        tmem_wait_ld16(v);
                    }
                    if (whole) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            *reinterpret_cast<uint4*>(stage + sw128(128, row, c / 8 + j)) =
                                make_uint4(bf16x2_bits(v[8 * j] * inv, v[8 * j + 1] * inv), bf16x2_bits(v[8 * j + 2] * inv, v[8 * j + 3] * inv),
                                           bf16x2_bits(v[8 * j + 4] * inv, v[8 * j + 5] * inv), bf16x2_bits(v[8 * j + 6] * inv, v[8 * j + 7] * inv));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<float4*>(stage + sw128(128, row, c / 4 + j)) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
                tc_fence_before();  // O is read before another product writes it
                __syncwarp();
                if (halves && lane == 0) mbar_arrive(read);
                const int chunks = whole ? cols / 8 : cols / 4;  // of a row, 16 bytes each: 4, 8, 16 or 32
                const int per = 32 / chunks, ch = lane & (chunks - 1);
#pragma unroll 4
                for (int i = 0; i < chunks; ++i) {
                    const int at = i * per + lane / chunks, lr = wrow + at, x = row0 + lr, xr = __shfl_sync(~0u, rel, at);
                    const uint4 w = *reinterpret_cast<const uint4*>(stage + sw128(128, lr, ch));
                    if (x >= nrows) continue;
                    if (whole) reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + (first_row + xr) * D + col0)[ch] = w;
                    else reinterpret_cast<uint4*>(part + (int64_t)x * D + col0)[ch] = w;
                }
                __syncwarp();
            };
            if (halves) put_out(mt * (D / 2), D / 2);
            else if (whole) put_out(0, D);
            else
                for (int half = 0; half < 2; ++half) put_out(half * (D / 2), D / 2);
            if (mine && (mt == 0 || !halves)) {
                if (!whole) *reinterpret_cast<float2*>(part + (int64_t)C::ROWS * D + 2 * r) = make_float2(m, l);
                else if (p.lse) p.lse[first_row + rel] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
            }
            if (!whole && y.kt0 == 0 && tid == 0) {
                desc->last = cta_of(all, ctas, walk.u - y.kt1 + y.kts - 1);
                desc->rows = nrows;
                desc->q0 = y.x.q0;
                desc->r0 = y.r0;
                desc->hk = y.hk;
            }
            if (halves) {  // the other warpgroup has read this one's O and statistics
                go = warp_wait(read, shared & 1);
                ++shared;
            }
        }
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

template <int D>
cudaError_t run(const Kv4AttentionParams& p, cudaStream_t s) {
    using C = Wide<D>;
    static std::atomic<uint64_t> ready{0};  // a bit for each device whose kernel attributes are set and checked
    const int sms = sm_count();
    if (sms == 0) return cudaErrorNoDevice;
    int dev = 0;
    CUtensorMap map;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = codes_map(p.kv, C::TILE, &map);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        // the warps' registers are split anew in the kernel: the block has to hold what that sums up to
        cudaFuncAttributes at{};
        e = cudaFuncGetAttributes(&at, gdn_kv4_attention_wide_kernel<C>);
        if (e != cudaSuccess) return e;
        if (at.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(gdn_kv4_attention_wide_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    gdn_kv4_attention_wide_kernel<C><<<sms, kThreads, C::SMEM, s>>>(p, map);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_kv4_join(p, C::ROWS, sms, s) : e;
}

}  // namespace

cudaError_t launch_kv4_attention_wide(const Kv4AttentionParams& p, cudaStream_t s) {
    return p.kv.D == 64 ? run<64>(p, s) : p.kv.D == 128 ? run<128>(p, s) : run<256>(p, s);
}

int64_t kv4_attention_wide_workspace(int D) {
    const int sms = sm_count();
    const int rows = D == 256 ? Wide<256>::ROWS : Wide<128>::ROWS;
    return (int64_t)(sms > 0 ? sms : 152) * ((int64_t)sizeof(PartDesc) + 2 * part_floats(rows, D) * 4);
}

}  // namespace gdn
