// gdn_kv4_attention.cu -- causal softmax attention of each lane's queries over its pages of the 4-bit cache.
//
//     o[t, h] = sum_j p_j v[j, h / G] / sum_j p_j,  p_j = exp(scale * q[t, h] . k[j, h / G] - max),
//     over the keys j <= kv_len - q_len + t of the lane;  lse[t, h] = max + log(sum_j p_j)
//
// The T tokens and the G = HQ / HK query heads of one key head are the rows of one product: row r is token r / G, head
// r % G, so the cached keys and values are read once for all of them.  An item is (lane, row tile, key head).
//
// Bound: the cache's 9/16 byte a number from HBM while an item has up to 16 rows; beyond that the tensor cores' rate for
// mma.sync (600 TFLOP/s measured).  Nothing is dequantised into memory: the packed tiles go to shared memory by
// cp.async (a pipeline of kStages tiles of 128 tokens), and each lane unpacks the codes of its own MMA fragments
// (cvt e2m1x2 -> f16x2, one multiply by the group's scale; both exact).  The products' summation index may be permuted
// freely, which makes the fragments contiguous in storage:
//   * S = Q K^T: lane (n, c) of a warp (n = lane / 4, c = lane % 4) supplies token n's dimensions; k step s takes
//     dimensions 4s .. 4s + 3 of the lane's own contiguous run, so one 16-byte load feeds 8 k steps.
//   * O = P V: lane (g, c) supplies dimension run g (D / 8 contiguous dimensions) of 4 tokens; column g of output tile i
//     is dimension g * D / 8 + i.  A pair of tokens is interleaved nibble by nibble before the conversion, so the f16x2
//     pairs come out as the MMA wants them, and their two scales multiply as one f16x2.
// P stays in registers: the accumulator layout of S is the A layout of P V.  Queries are scaled to f16 by a power of two
// a row (exact but for values 2^-14 below the row's largest); P is rounded to f16 (half a step 2^-12 of a value in
// 0 .. 1, well below the bf16 rounding of o), the sums l are those of the unrounded P in fp32, as all statistics are.
//
// Work split: all tiles of all items are numbered item by item and each CTA takes an equal run of them, so one long lane
// fills the GPU as well as many short ones.  A run ends in an item's middle on most CTAs: such parts (m, l, O in fp32) go
// to the workspace, two at most a CTA, and a second kernel, launched programmatically behind the first, joins them in
// order.  The four warps of a CTA take 32 tokens each of a tile, or with more than kMT * 16 rows half the warps take
// other rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// MT: m16 row tiles of a warp; WR: warps side by side along the rows; the other kWarps / WR share a tile's tokens
template <int D_, int MT_, int WR_>
struct Cfg {
    static constexpr int D = D_, MT = MT_, WR = WR_, WK = kWarps / WR;
    static constexpr int ROWS = 16 * MT * WR;      // of an item
    static constexpr int WT = D == 256 ? 16 : 32;  // tokens of a warp's step
    static constexpr int KT = 128;                 // tokens of a tile
    static constexpr int STEPS = KT / (WT * WK);   // steps of a warp in a tile
    static constexpr int STAGES = D == 256 ? 2 : 3;
    static constexpr int CB = D / 2, SB = D / 16;  // bytes of a token's codes and scales
    static constexpr int STAGE = 2 * KT * (CB + SB);
    static constexpr int QFRAG = ROWS / 16 * (D / 16) * 512;  // Q as MMA fragments
    static constexpr int MERGE = WK * ROWS * D * 4;           // the warps' O before they are joined
    static constexpr int POOL = STAGES * STAGE > MERGE ? STAGES * STAGE : MERGE;
    static constexpr int SMEM = POOL + QFRAG + WK * ROWS * 8 + ROWS * 4;
    static_assert(STEPS * WT * WK == KT, "tile split");
};

// Byte offset of 16-byte chunk c of token row r in a tile of codes: chunks XORed so that the fragment loads of K (rows
// 2j, 2j+1 together) and of V (rows 0, 3, 4, 7 or 1, 2, 5, 6 together) meet no bank twice
template <int D>
__device__ __forceinline__ int code_off(int r, int c) {
    if (D == 64) return r * 32 + c * 16;
    if (D == 128) return r * 64 + ((c ^ (((r >> 2) & 1) << 1)) << 4);
    return r * 128 + ((c ^ (((r & 1) << 2) ^ (((r >> 2) & 1) << 1))) << 4);
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

struct Item {
    int b, rt, hk;
    int q0, qlen, kv;  // the lane's first row in q, tokens, cached tokens
};

// One lane's extent; qlen 0: nothing to do
__device__ __forceinline__ void lane_extent(const Kv4AttentionParams& p, int b, int& q0, int& qlen, int& kv, uint32_t& bits) {
    int64_t a = (int64_t)b * p.T, n = p.T;
    if (p.cu_seqlens) {
        a = p.cu_seqlens[b];
        n = (int64_t)p.cu_seqlens[b + 1] - a;
    }
    kv = p.kv_lens[b];
    q0 = (int)a;
    qlen = (int)n;
    if (a < 0 || n < 0 || n > p.T || a + n > p.N || kv < 0 || kv > (int64_t)p.max_pages * p.kv.page_size) {
        bits |= GDN_ERRBIT_SEQLEN;
        qlen = 0;
    }
}

template <typename C>
__global__ void __launch_bounds__(kThreads) gdn_kv4_attention_kernel(Kv4AttentionParams p) {
    constexpr int D = C::D, MT = C::MT, KT = C::KT, WT = C::WT;
    constexpr int KS = D / 16;          // k steps of S
    constexpr int NT = WT / 8;          // token groups of 8
    constexpr int DT = D / 8;           // output tiles of 8 columns
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_scan[kThreads + 1];
    uint8_t* pool = smem;
    uint4* s_q = reinterpret_cast<uint4*>(smem + C::POOL);
    float2* s_ml = reinterpret_cast<float2*>(smem + C::POOL + C::QFRAG);             // [WK][ROWS]
    float* s_sc = reinterpret_cast<float*>(smem + C::POOL + C::QFRAG + C::WK * C::ROWS * 8);  // [ROWS]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int wr = warp % C::WR, wk = warp / C::WR;
    const uint32_t pool_u = smem_u32(pool);
    uint32_t bits = 0;
    float* parts = reinterpret_cast<float*>(reinterpret_cast<PartDesc*>(p.workspace) + gridDim.x);
    const int HK = p.kv.HK, P = p.kv.page_size, pshift = 31 - __clz(P);

    // ---- this CTA's run of tiles --------------------------------------------------------------------------
    const int per = (p.B + kThreads - 1) / kThreads;
    auto lane_tiles = [&](int b) -> int64_t {
        int q0, qlen, kv;
        lane_extent(p, b, q0, qlen, kv, bits);
        const int64_t rts = ((int64_t)qlen * p.G + C::ROWS - 1) / C::ROWS;
        const int64_t kts = kv > 0 ? (kv + KT - 1) / KT : 1;
        return rts * kts * HK;
    };
    {
        int64_t mine = 0;
        for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) mine += lane_tiles(b);
        int64_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_scan[kThreads - 3 + warp] = x;  // the last places are free until the sums are in
        __syncthreads();
        int64_t before = 0;
        for (int w = 0; w < warp; ++w) before += s_scan[kThreads - 3 + w];
        __syncthreads();
        s_scan[tid + 1] = before + x;
        if (tid == 0) s_scan[0] = 0;
        __syncthreads();
    }
    const int64_t all = s_scan[kThreads];
    const int64_t ctas = all < gridDim.x ? all : gridDim.x;
    const int64_t u0 = blockIdx.x < ctas ? all * blockIdx.x / ctas : all, u1 = blockIdx.x < ctas ? all * (blockIdx.x + 1) / ctas : all;
    PartDesc* desc = reinterpret_cast<PartDesc*>(p.workspace) + blockIdx.x;
    if (tid == 0) desc->last = -1;
    if (bits && p.err && blockIdx.x == 0) atomicOr(p.err, (int32_t)bits);
    bits = 0;

    int b = 0;
    int64_t base = 0;  // first tile of lane b
    if (u0 < u1) {
        int lo = 0, hi = kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_scan[mid] <= u0) lo = mid;
            else hi = mid;
        }
        b = lo * per;
        base = s_scan[lo];
    }
    for (int64_t u = u0; u < u1;) {
        // the item that holds tile u
        int64_t n = lane_tiles(b);
        while (base + n <= u) {
            base += n;
            n = lane_tiles(++b);
        }
        int q0, qlen, kv;
        lane_extent(p, b, q0, qlen, kv, bits);
        const int kts = kv > 0 ? (kv + KT - 1) / KT : 1;
        const int64_t in = u - base;
        const int item = (int)(in / kts), kt0 = (int)(in - (int64_t)item * kts);
        const int hk = item % HK, rt = item / HK, r0 = rt * C::ROWS;
        const int nrows = min(C::ROWS, qlen * p.G - r0);
        const int kt1 = (int)min((int64_t)kts, kt0 + (u1 - u));
        const int64_t u_item = u - kt0;  // the item's first tile
        const int32_t* table = p.block_tables + (int64_t)b * p.max_pages;

        // ---- the pipeline of tiles: thread i copies chunks of the token rows i / (CB / 16) + k * ROWSTEP -------
        constexpr int CPR = C::CB / 16, RSTEP = kThreads / CPR, NR = KT / RSTEP;  // chunks of a row; rows a pass; passes
        constexpr int SCH = KT * C::SB / 16;                                      // chunks of a tile's K (or V) scales
        const int crow = tid / CPR, cch = tid % CPR;
        auto page_of = [&](int tok) -> int {
            if (tok >= kv) return -1;
            const int pg = table[tok >> pshift];
            if ((uint32_t)pg >= (uint32_t)p.kv.num_pages) {
                bits |= GDN_ERRBIT_INDEX;
                return -1;
            }
            return pg;
        };
        int pg[NR], spg[2];
        auto fetch_pages = [&](int kt) {
#pragma unroll
            for (int i = 0; i < NR; ++i) pg[i] = kt < kt1 ? page_of(kt * KT + crow + i * RSTEP) : -1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ch = tid + i * kThreads;
                const int tok = kt * KT + (ch % SCH) * (16 / C::SB);
                spg[i] = ch < 2 * SCH && kt < kt1 ? page_of(tok) : -1;
            }
        };
        auto issue = [&](int kt) {  // from the pages that fetch_pages(kt) found
            if (kt < kt1) {
                const uint32_t st = pool_u + (uint32_t)((kt - kt0) % C::STAGES) * C::STAGE;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int r = crow + i * RSTEP, off = (kt * KT + r) & (P - 1);
                    const int64_t row = ((int64_t)max(pg[i], 0) * 2 * HK + hk) * P + off;
                    const uint8_t* src = p.kv.codes + row * C::CB + cch * 16;
                    const uint32_t n16 = pg[i] >= 0 ? 16u : 0u;
                    cp_async16(st + code_off<D>(r, cch), src, n16);
                    cp_async16(st + KT * C::CB + code_off<D>(r, cch), src + (int64_t)HK * P * C::CB, n16);
                }
#pragma unroll
                for (int i = 0; i < (2 * SCH + kThreads - 1) / kThreads; ++i) {
                    const int ch = tid + i * kThreads;
                    if (ch < 2 * SCH) {
                        const int which = ch / SCH, r = (ch % SCH) * (16 / C::SB), off = (kt * KT + r) & (P - 1);
                        const int64_t row = (((int64_t)max(spg[i], 0) * 2 + which) * HK + hk) * P + off;
                        // tokens that end inside the chunk leave zero scales behind them, whatever the page holds
                        const int n = spg[i] >= 0 ? min(16, (kv - kt * KT - r) * C::SB) : 0;
                        cp_async16(st + 2 * KT * C::CB + ch * 16, p.kv.scales + row * C::SB, (uint32_t)n);
                    }
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < C::STAGES - 1; ++s) {
            fetch_pages(kt0 + s);
            issue(kt0 + s);
        }
        fetch_pages(kt0 + C::STAGES - 1);

        // ---- Q as f16 fragments in shared memory, each row scaled by a power of two -----------------------------
        for (int r = warp; r < C::ROWS; r += kWarps) {
            float x[D / 32];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint32_t w = 0;
                if (r < nrows) {
                    const int t = (r0 + r) / p.G, h = hk * p.G + (r0 + r) - t * p.G;
                    w = *reinterpret_cast<const uint32_t*>((const __nv_bfloat16*)p.q + ((int64_t)(q0 + t) * p.HQ + h) * D + i * 64 + lane * 2);
                }
                x[2 * i] = __uint_as_float(w << 16);
                x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            // top's power of two, kept where it and its reciprocal are normal numbers
            uint32_t e = __float_as_uint(top) >> 23;
            e = e < 30 ? 30 : e > 224 ? 224 : e;
            const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
            if (lane == 0) s_sc[r] = up * p.scale * p.kv.k_scale * kLog2e;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                // dimension d is part of lane c's run: for D 128 c = d / 32 and k step (d % 32) / 4; for 64 runs of 16;
                // for 256 two halves of 128
                const int d = i * 64 + lane * 2;
                constexpr int RUN = D == 64 ? 16 : 32;
                const int half = D == 256 ? d >> 7 : 0, dd = D == 256 ? d & 127 : d;
                const int cc = dd / RUN, ks = half * (RUN / 4) + (dd % RUN) / 4, pair = (dd % 4) / 2;
                const int mt = r / 16, rr = r % 16;
                // fragment words: a0 (row g, pair 0), a1 (row g + 8, pair 0), a2 (row g, pair 1), a3 (row g + 8, pair 1)
                uint32_t* f = reinterpret_cast<uint32_t*>(s_q + (mt * KS + ks) * 32 + (rr % 8) * 4 + cc);
                f[pair * 2 + rr / 8] = f16x2_bits(x[2 * i] * down, x[2 * i + 1] * down);
            }
        }
        __syncthreads();

        float o[MT][DT][4], m[MT][2], l[MT][2], sc[MT][2];
        int limit[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = (wr * MT + mt) * 16 + h * 8 + g;
                m[mt][h] = -INFINITY;
                l[mt][h] = 0.f;
                sc[mt][h] = s_sc[r];
                limit[mt][h] = kv - qlen + (r0 + r) / p.G + 1;  // keys that the row sees
#pragma unroll
                for (int i = 0; i < DT; ++i) o[mt][i][2 * h] = o[mt][i][2 * h + 1] = 0.f;
            }
        const int all_see = kv - qlen + r0 / p.G + 1;  // keys that every row sees

        for (int kt = kt0; kt < kt1; ++kt) {
            cp_async_wait<C::STAGES - 2>();
            __syncthreads();
            issue(kt + C::STAGES - 1);
            fetch_pages(kt + C::STAGES);
            const uint8_t* st = pool + (size_t)((kt - kt0) % C::STAGES) * C::STAGE;
            const uint8_t *kc = st, *vc = st + KT * C::CB, *ksc = st + 2 * KT * C::CB, *vsc = ksc + KT * C::SB;
#pragma unroll 1
            for (int step = 0; step < C::STEPS; ++step) {
                const int w0 = (step * C::WK + wk) * WT;  // the warp's first token in the tile
                // S: token group j's column n is token j * 8 + (n ^ ((n >> 1) & 1))
                float s[MT][NT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[mt][j][i] = 0.f;
#pragma unroll
                for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
                    uint32_t w[NT][D == 64 ? 2 : 4], scl[NT][2];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int r = w0 + j * 8 + (g ^ ((g >> 1) & 1));
                        if constexpr (D == 64) {
                            const uint2 v = *reinterpret_cast<const uint2*>(kc + r * 32 + c * 8);
                            w[j][0] = v.x;
                            w[j][1] = v.y;
                            const uint32_t f = e4m3x2_to_f16(ksc[r * 4 + c] * 0x101u);
                            scl[j][0] = scl[j][1] = f;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(kc + code_off<D>(r, half * 4 + c));
                            w[j][0] = v.x;
                            w[j][1] = v.y;
                            w[j][2] = v.z;
                            w[j][3] = v.w;
                            const uint32_t f = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(ksc + r * C::SB + half * 8 + c * 2));
                            scl[j][0] = __byte_perm(f, f, 0x1010);
                            scl[j][1] = __byte_perm(f, f, 0x3232);
                        }
                    }
                    constexpr int WN = D == 64 ? 2 : 4;
#pragma unroll
                    for (int i = 0; i < WN; ++i) {
                        uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const uint4* q = s_q + ((wr * MT + mt) * KS + half * 8 + 2 * i) * 32 + lane;
                            const uint4 x = q[0], y = q[32];
                            a0[mt][0] = x.x, a0[mt][1] = x.y, a0[mt][2] = x.z, a0[mt][3] = x.w;
                            a1[mt][0] = y.x, a1[mt][1] = y.y, a1[mt][2] = y.z, a1[mt][3] = y.w;
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            uint32_t f[4];
                            e2m1x8_to_f16(w[j][i], f);
                            const uint32_t sf = scl[j][i / 2];
#pragma unroll
                            for (int x = 0; x < 4; ++x) f[x] = hmul2(f[x], sf);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma_f16(s[mt][j], a0[mt], f[0], f[1]);
                                mma_f16(s[mt][j], a1[mt], f[2], f[3]);
                            }
                        }
                    }
                }
                // softmax in units of log 2
                const int tok0 = kt * KT + w0;
                uint32_t pf[MT][NT][2];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int h = i >> 1, n = 2 * c + (i & 1);
                            float x = s[mt][j][i] * sc[mt][h];
                            if (tok0 + WT > all_see && tok0 + j * 8 + (n ^ (c & 1)) >= limit[mt][h]) x = -INFINITY;
                            s[mt][j][i] = x;
                            top[h] = fmaxf(top[h], x);
                        }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        top[h] = fmaxf(top[h], __shfl_xor_sync(~0u, top[h], 1));
                        top[h] = fmaxf(top[h], __shfl_xor_sync(~0u, top[h], 2));
                    }
                    if (__any_sync(~0u, top[0] > m[mt][0] || top[1] > m[mt][1])) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float mn = fmaxf(m[mt][h], top[h]);
                            const float f = mn == -INFINITY ? 1.f : exp2_fast(m[mt][h] - mn);
                            m[mt][h] = mn;
                            l[mt][h] *= f;
#pragma unroll
                            for (int i = 0; i < DT; ++i) {
                                o[mt][i][2 * h] *= f;
                                o[mt][i][2 * h + 1] *= f;
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mm = m[mt][h] == -INFINITY ? 0.f : m[mt][h];
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const float e0 = exp2_fast(s[mt][j][2 * h] - mm), e1 = exp2_fast(s[mt][j][2 * h + 1] - mm);
                            l[mt][h] += e0 + e1;
                            pf[mt][j][h] = f16x2_bits(e0, e1);
                        }
                    }
                }
                // O += P V: 16 tokens at a time; this lane's tokens are 2c, 2c + 1 of two groups, swapped for odd c
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    constexpr int WN = D / 64;  // words of a run of D / 8 dimensions
                    uint32_t w[4][WN], sv[2][WN > 2 ? 2 : 1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 2 * c + (i & 1), r = w0 + (j + (i >> 1)) * 8 + (n ^ (c & 1));
                        if constexpr (D == 64) {
                            w[i][0] = *reinterpret_cast<const uint32_t*>(vc + r * 32 + g * 4);
                        } else if constexpr (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(vc + code_off<D>(r, g >> 1) + (g & 1) * 8);
                            w[i][0] = v.x;
                            w[i][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(vc + code_off<D>(r, g));
                            w[i][0] = v.x;
                            w[i][1] = v.y;
                            w[i][2] = v.z;
                            w[i][3] = v.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int ra = w0 + (j + i) * 8 + ((2 * c) ^ (c & 1)), rb = w0 + (j + i) * 8 + ((2 * c + 1) ^ (c & 1));
                        if constexpr (D == 256) {
                            const uint32_t x = *reinterpret_cast<const uint16_t*>(vsc + ra * 16 + g * 2);
                            const uint32_t y = *reinterpret_cast<const uint16_t*>(vsc + rb * 16 + g * 2);
                            sv[i][0] = e4m3x2_to_f16(__byte_perm(x, y, 0x0040));
                            sv[i][1] = e4m3x2_to_f16(__byte_perm(x, y, 0x0051));
                        } else {
                            const int gr = D == 64 ? g >> 1 : g;
                            sv[i][0] = e4m3x2_to_f16((uint32_t)vsc[ra * C::SB + gr] | ((uint32_t)vsc[rb * C::SB + gr] << 8));
                        }
                    }
                    uint32_t pa[MT][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        pa[mt][0] = pf[mt][j][0];
                        pa[mt][1] = pf[mt][j][1];
                        pa[mt][2] = pf[mt][j + 1][0];
                        pa[mt][3] = pf[mt][j + 1][1];
                    }
#pragma unroll
                    for (int x = 0; x < WN; ++x) {
                        // bytes (token a, token b) of one dimension: even dimensions, then odd ones
                        uint32_t f[2][2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t wa = w[2 * i][x], wb = w[2 * i + 1][x];
                            e2m1x8_to_f16((wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u), f[i][0]);
                            e2m1x8_to_f16(((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u), f[i][1]);
                            const uint32_t sf = sv[i][D == 256 ? x / 2 : 0];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                f[i][0][y] = hmul2(f[i][0][y], sf);
                                f[i][1][y] = hmul2(f[i][1][y], sf);
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 8; ++y)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma_f16(o[mt][x * 8 + y], pa[mt], f[0][y & 1][y >> 1], f[1][y & 1][y >> 1]);
                    }
                }
            }
        }
        cp_async_wait<0>();
        __syncthreads();

        // ---- the warps' parts of the item joined, then stored ----------------------------------------------------
        float* s_o = reinterpret_cast<float*>(pool);  // [WK][ROWS][D]
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = l[mt][h];
                x += __shfl_xor_sync(~0u, x, 1);
                x += __shfl_xor_sync(~0u, x, 2);
                const int r = (wr * MT + mt) * 16 + h * 8 + g;
                if (c == 0) s_ml[wk * C::ROWS + r] = make_float2(m[mt][h], x);
                float* dst = s_o + ((size_t)wk * C::ROWS + r) * D;
#pragma unroll
                for (int i = 0; i < DT; ++i) {
                    dst[(2 * c) * (D / 8) + i] = o[mt][i][2 * h];
                    dst[(2 * c + 1) * (D / 8) + i] = o[mt][i][2 * h + 1];
                }
            }
        __syncthreads();
        const bool whole = kt0 == 0 && kt1 == kts;
        float* part = parts + ((int64_t)blockIdx.x * 2 + (kt0 == 0 ? 1 : 0)) * part_floats(C::ROWS, D);
        for (int r = warp; r < nrows; r += kWarps) {
            float mm = -INFINITY, ll = 0.f, f[C::WK];
#pragma unroll
            for (int w = 0; w < C::WK; ++w) mm = fmaxf(mm, s_ml[w * C::ROWS + r].x);
#pragma unroll
            for (int w = 0; w < C::WK; ++w) {
                const float2 x = s_ml[w * C::ROWS + r];
                f[w] = mm == -INFINITY ? 1.f : exp2_fast(x.x - mm);
                ll += x.y * f[w];
            }
            const int t = (r0 + r) / p.G, h = hk * p.G + (r0 + r) - t * p.G;
            const int64_t out = (int64_t)(q0 + t) * p.HQ + h;
            const float inv = ll > 0.f ? p.kv.v_scale / ll : ll != ll ? ll : 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int d = i * 64 + lane * 2;
                float a = 0.f, bb = 0.f;
#pragma unroll
                for (int w = 0; w < C::WK; ++w) {
                    const float2 x = *reinterpret_cast<const float2*>(s_o + ((size_t)w * C::ROWS + r) * D + d);
                    a = fmaf(x.x, f[w], a);
                    bb = fmaf(x.y, f[w], bb);
                }
                if (whole) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(a * inv, bb * inv);
                    *reinterpret_cast<__nv_bfloat162*>((__nv_bfloat16*)p.o + out * D + d) = y;
                } else {
                    *reinterpret_cast<float2*>(part + (int64_t)r * D + d) = make_float2(a, bb);
                }
            }
            if (lane == 0) {
                if (whole) {
                    if (p.lse) p.lse[out] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
                } else {
                    part[(int64_t)C::ROWS * D + 2 * r] = mm;
                    part[(int64_t)C::ROWS * D + 2 * r + 1] = ll;
                }
            }
        }
        if (!whole && kt0 == 0 && tid == 0) {
            // the CTA whose run holds the item's last tile
            const int64_t end = u_item + kts - 1;
            int64_t z = (end * ctas) / all;
            while (all * (z + 1) / ctas <= end) ++z;
            while (all * z / ctas > end) --z;
            desc->last = (int32_t)z;
            desc->rows = nrows;
            desc->q0 = q0;
            desc->r0 = r0;
            desc->hk = hk;
        }
        __syncthreads();
        u += kt1 - kt0;
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);
}

// Joins the parts of the items that CTA x of the first kernel began and did not end: block (x, y) takes rows y, y + gridDim.y, ..
template <typename C>
__global__ void __launch_bounds__(kThreads) gdn_kv4_attention_join_kernel(Kv4AttentionParams p, int ctas) {
    constexpr int D = C::D;
    grid_dependency_wait();
    const PartDesc d = reinterpret_cast<const PartDesc*>(p.workspace)[blockIdx.x];
    if (d.last < 0) return;
    const float* parts = reinterpret_cast<const float*>(reinterpret_cast<const PartDesc*>(p.workspace) + ctas);
    const int first = blockIdx.x, n = d.last - first + 1;
    const int64_t step = part_floats(C::ROWS, D);
    for (int r = blockIdx.y; r < d.rows; r += gridDim.y) {
        auto part = [&](int i) { return parts + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * step; };
        float mm = -INFINITY;
        for (int i = 0; i < n; ++i) mm = fmaxf(mm, part(i)[(int64_t)C::ROWS * D + 2 * r]);
        float ll = 0.f, a[(D + kThreads - 1) / kThreads] = {};
        for (int i = 0; i < n; ++i) {
            const float* q = part(i);
            const float f = mm == -INFINITY ? 1.f : exp2_fast(q[(int64_t)C::ROWS * D + 2 * r] - mm);
            ll = fmaf(q[(int64_t)C::ROWS * D + 2 * r + 1], f, ll);
#pragma unroll
            for (int k = 0; k < (D + kThreads - 1) / kThreads; ++k) {
                const int x = threadIdx.x + k * kThreads;
                if (x < D) a[k] = fmaf(q[(int64_t)r * D + x], f, a[k]);
            }
        }
        const int t = (d.r0 + r) / p.G, h = d.hk * p.G + (d.r0 + r) - t * p.G;
        const int64_t out = (int64_t)(d.q0 + t) * p.HQ + h;
        const float inv = ll > 0.f ? p.kv.v_scale / ll : ll != ll ? ll : 0.f;
#pragma unroll
        for (int k = 0; k < (D + kThreads - 1) / kThreads; ++k) {
            const int x = threadIdx.x + k * kThreads;
            if (x < D) ((__nv_bfloat16*)p.o)[out * D + x] = __float2bfloat16_rn(a[k] * inv);
        }
        if (threadIdx.x == 0 && p.lse) p.lse[out] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
    }
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

constexpr int kCtasPerSm = 2;

template <typename C>
cudaError_t run(const Kv4AttentionParams& p, cudaStream_t s) {
    const int sms = sm_count();
    if (sms == 0) return cudaErrorNoDevice;
    const int ctas = sms * kCtasPerSm;
    cudaError_t e = cudaFuncSetAttribute(gdn_kv4_attention_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    gdn_kv4_attention_kernel<C><<<ctas, kThreads, C::SMEM, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, C::ROWS < 8 ? C::ROWS : 8);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_kv4_attention_join_kernel<C>, p, ctas);
}

// Rows of an item: one m16 tile a warp while the lane's rows fit it, two up to 32 (a warp's unpacked fragments then serve
// both); more rows go to other warps.  D = 256 keeps one (its O takes 128 registers a thread).
int item_rows(int64_t rows, int D) {
    if (rows <= 16) return 16;
    if (rows <= 32) return 32;
    return 64;
}

template <int D>
cudaError_t run_d(const Kv4AttentionParams& p, int rows, cudaStream_t s) {
    if constexpr (D == 256) {
        return rows == 16 ? run<Cfg<256, 1, 1>>(p, s) : rows == 32 ? run<Cfg<256, 1, 2>>(p, s) : run<Cfg<256, 1, 4>>(p, s);
    } else {
        return rows == 16 ? run<Cfg<D, 1, 1>>(p, s) : rows == 32 ? run<Cfg<D, 2, 1>>(p, s) : run<Cfg<D, 2, 2>>(p, s);
    }
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttentionParams& p, cudaStream_t s) {
    const int rows = item_rows((int64_t)p.T * p.G, p.kv.D);
    return p.kv.D == 64    ? run_d<64>(p, rows, s)
           : p.kv.D == 128 ? run_d<128>(p, rows, s)
                           : run_d<256>(p, rows, s);
}

int64_t kv4_attention_workspace(int B, int T, int HQ, int HK, int D) {
    (void)B;
    const int sms = sm_count();
    const int64_t ctas = (int64_t)(sms > 0 ? sms : 152) * kCtasPerSm;
    const int rows = item_rows((int64_t)T * (HQ / HK), D);
    return ctas * ((int64_t)sizeof(PartDesc) + 2 * part_floats(rows, D) * 4);
}

}  // namespace gdn
