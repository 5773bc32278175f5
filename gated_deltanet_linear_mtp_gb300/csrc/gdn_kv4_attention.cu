// gdn_kv4_attention.cu -- causal softmax attention of each lane's queries over its pages of the 4-bit cache.
//
//     o[t, h] = sum_j p_j v[j, h / G] / sum_j p_j,  p_j = exp(scale * q[t, h] . k[j, h / G] - max),
//     over the keys j <= kv_len - q_len + t of the lane;  lse[t, h] = max + log(sum_j p_j)
//
// The T tokens and the G = HQ / HK query heads of one key head are the rows of one product: row r is token r / G, head
// r % G, so the cached keys and values are read once for all of them.  An item is (lane, row tile, key head).
//
// Floor: the cache's 9/16 byte a number from HBM.  Measured with the join (graph replays, HBM's floor in brackets): one lane of 131071
// tokens, HQ 32, HK 4, D 128, 28 us (11); 64 lanes of one token over up to 8192, HQ 16, HK 2, D 256, 48 us (23), 3.3 TB/s; 128 lanes
// of 4 tokens over up to 16384, HQ 32, HK 4, D 128, 307 us (94), 230 TFLOP/s; the same with HQ 16, HK 2, D 256, whose 32 rows are
// two items that each read the cache, 319 us (94).  What lies above: nothing is full (128 lanes of 4: issue slots 44 %, the tensor
// pipe 39 %, DRAM 26 %).  Each of the two computing warps of a scheduler runs unpacking (two conversions' worth of instructions a
// pair of numbers), S, softmax and P V one after the other, and O's registers leave no place for a third.  More rows go to
// gdn_kv4_attention_wide.cu.
// Nothing is dequantised into memory: one warp brings packed tiles of 128 or 256 tokens into shared memory by TMA (swizzled, a
// pipeline of several), and each lane of the others unpacks the codes of its own MMA fragments (cvt e2m1x2 -> f16x2, one
// multiply by the group's scale; both exact).  Issue: an eighth of a tile costs a warp about 760 instructions at 32 rows, D 128
// (16 warps of half the rows each were not faster: 396 us against 371 then).  Keys and values are the M operand and the rows are N:
// N goes by 8, so a decode's 8 rows waste nothing.  The products' summation index may be permuted freely, which makes the
// fragments contiguous in storage:
//   * S^T = K Q^T: lane (g, c) of a warp (g = lane / 4, c = lane % 4) supplies tokens g and g + 8 of a tile of 16; k step s
//     takes dimensions 4s .. 4s + 3 of the lane's own contiguous run, so one 16-byte load feeds 8 k steps.
//   * O^T = V^T P^T: lane (g, c) supplies dimension run g (D / 8 contiguous dimensions) of 4 tokens; rows g and g + 8 of
//     output tile i are dimensions 2i and 2i + 1 of that run.  A pair of tokens is interleaved nibble by nibble before the
//     conversion, so the f16x2 pairs come out as the MMA wants them, and their two scales multiply as one f16x2.
// P goes from accumulator to operand layout by one movmatrix for each 8 x 8.  Queries are scaled to f16 by a power of two
// a row (exact but for values 2^-14 below the row's largest); P is rounded to f16 (half a step 2^-11 of a value, well
// below the bf16 rounding of o; 2^-32 of the row's largest at least, by kLift), the sums l are those of the unrounded P in
// fp32, as all statistics are.  The reference m is moved only where a score passes it by more than kLift + 8 (in units of log
// 2), so most steps need no exchange between lanes.
//
// Work split: all tiles of all items are numbered item by item and each CTA takes an equal run of them, so one long lane
// fills the GPU as well as many short ones.  A run ends in an item's middle on most CTAs: such parts (m, l, O in fp32) go
// to the workspace, two at most a CTA, and a second kernel, launched programmatically behind the first, joins them in
// order.  The eight warps of a CTA take 16 or 32 tokens each of a tile and join their parts in shared memory.
#include <algorithm>
#include <atomic>

#include "gdn_kv4_attention.cuh"

namespace gdn {

namespace {

// NR: groups of 8 rows of an item; W: warps that compute (one of four more copies, and those four give their registers to
// the others: LREG a thread at launch, then CREG and PREG); WT: tokens of a warp's step; TILE: tokens of a tile; STAGES: tiles
// in the pipeline; CTAS: of an SM; SWITCH: tiles that an item's begin and end (queries in, the warps' parts joined) count as in
// the split of the work, so that CTAs with many short items are done with the others.  Readings in us with 0, 1, 2, 3, 4, 5, 6, 8
// (* the one taken), ragged contexts up to the given one, HQ 32 and HK 4, at D 256 16 and 2:
//   D 64,  8 rows,  64 lanes, 8192:   39* 36 37 38 39 41 41 43 (of another batch of lanes 92* 97 with 0 and 1)
//   D 64,  16 rows, 128 lanes, 8192:  86 76* 72 72 72 74 76 78
//   D 64,  32 rows, 128 lanes, 16384: 259 254 248 244* 235 230 222 215;  64 lanes, 4096: 62 60 58 55* 51 49 47 49
//   D 128, 8 rows,  64 lanes, 8192:   53 48 49* 49 51 54 53 57
//   D 128, 16 rows, 128 lanes, 8192:  135 119 111 109* 111 112 115 117
//   D 128, 32 rows, 128 lanes, 16384: 361 354 345 337 323 314 306* 312
//   D 256, 8 rows,  64 lanes, 8192:   54 51 49 47* 49 49 50 52
//   D 256, 16 rows, 128 lanes, 8192:  121 111 106 103 99 100* 102 103;  32 rows, 16384: 361 347 338 328 318 319* 321 328
// At D 64 a larger one reads better with 32 rows (12 %) and with 16 (6 %).
template <int D_, int NR_, int WT_, int TILE_, int STAGES_, int CTAS_, int SWITCH_>
struct Cfg {
    static constexpr int D = D_, NR = NR_, W = 8, WT = WT_, TILE = TILE_, STAGES = STAGES_, CTAS = CTAS_;
    static constexpr bool SPLIT = false;  // a stage holds keys and values
    static constexpr int SWITCH = SWITCH_;
    static constexpr int ROWS = 8 * NR, THREADS = 32 * (W + 4), STEPS = TILE / W / WT;
    static constexpr int CB = D / 2, SB = D / 16;  // bytes of a token's codes and scales
    static constexpr int STAGE = 2 * TILE * (CB + SB);
    static constexpr bool QREG = D / 8 * NR <= 32;  // Q's fragments stay in registers
    static constexpr int QBYTES = ROWS * D * 2;
    static constexpr int OROW = D + 4;  // floats of a row while the warps' parts are joined
    static constexpr int MERGE = W * 8 * OROW * 4;
    static constexpr int SMEM = 1024 + STAGES * STAGE + QBYTES + MERGE + W * 64 + ROWS * 4;
    static constexpr int LREG = CTAS == 1 ? 168 : 80, CREG = CTAS == 1 ? 232 : 104, PREG = CTAS == 1 ? 40 : 32;
    static_assert(2 * CREG + PREG <= 3 * LREG, "the block's registers");
    static_assert(STEPS * W * WT == TILE && TILE % 128 == 0 && WT % 16 == 0, "tile split");
};

// The reference of a row that has seen no key: below any score, and finite, so that a masked score's -inf less it is -inf without
// a test (64 lanes of one token, HQ 16, HK 2, D 256: 47.7 us against 49.2 with -inf and the test)
constexpr float kNone = -3.402823466e38f;

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

template <typename C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS) gdn_kv4_attention_kernel(const __grid_constant__ Kv4AttentionParams p,
                                                                     const __grid_constant__ CUtensorMap map) {
    constexpr int D = C::D, NR = C::NR, WT = C::WT;
    constexpr int KS = D / 16;   // k steps of S
    constexpr int NT = WT / 8;   // groups of 8 tokens of a step
    constexpr int DT = D / 16;   // output tiles of 16 dimensions
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t s_scan[C::THREADS + 1];
    __shared__ int64_t s_warp[C::W + 4];
    __shared__ uint64_t s_bar[2 * C::STAGES];
    __shared__ int s_dead;
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* pool = smem;
    uint4* s_q = reinterpret_cast<uint4*>(smem + C::STAGES * C::STAGE);
    float* s_o = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE + C::QBYTES);  // [W][8][OROW]
    float2* s_ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(s_o) + C::MERGE);  // [W][8]
    float* s_sc = reinterpret_cast<float*>(s_ml + C::W * 8);                             // [ROWS]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t full = smem_u32(s_bar), empty = full + 8 * C::STAGES;
    uint32_t bits = 0;

    // ---- this CTA's run of tiles --------------------------------------------------------------------------
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, C::W);
        }
        fence_mbar_init();
        s_dead = 0;
    }
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    scan_lanes<C>(p, per, s_scan, s_warp, bits);
    const int64_t all = s_scan[C::THREADS], ctas = all < gridDim.x ? all : gridDim.x;
    PartDesc* desc = reinterpret_cast<PartDesc*>(p.workspace) + blockIdx.x;
    float* parts = reinterpret_cast<float*>(reinterpret_cast<PartDesc*>(p.workspace) + gridDim.x);
    if (tid == 0) desc->last = -1;
    if (bits && p.err && blockIdx.x == 0) atomicOr(p.err, (int32_t)bits);
    bits = 0;
    if (blockIdx.x >= ctas) return;
    Walk<C> walk = begin_walk<C>(per, s_scan, all, ctas);
    if (warp >= C::W) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::PREG));
        if (warp > C::W) return;
        produce<C>(p, &map, walk, smem_u32(pool), pool, full, empty, bits);
        if (bits && p.err) atomicOr(p.err, (int32_t)bits);
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::CREG));
    uint32_t it = 0;
    bool dead = false;
    Piece y;
    while (walk.next(p, y)) {
        const int nrows = min(C::ROWS, y.x.qlen * p.G - y.r0);
        // ---- Q as f16 fragments in shared memory, each row scaled by a power of two ---------------------------
        for (int r = warp; r < C::ROWS; r += C::W) {
            float x[D / 32];
            float top = 0.f;
            const int t = (y.r0 + r) / p.G, h = y.hk * p.G + (y.r0 + r) - t * p.G;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint32_t w = 0;
                if (r < nrows)
                    w = *reinterpret_cast<const uint32_t*>((const __nv_bfloat16*)p.q + ((int64_t)(y.x.q0 + t) * p.HQ + h) * D +
                                                           i * 64 + lane * 2);
                x[2 * i] = __uint_as_float(w << 16);
                x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const uint32_t e = row_exponent(__float_as_uint(top) >> 23);
            const float down = __uint_as_float((254u - e) << 23);
            if (lane == 0) s_sc[r] = row_scale(p, e, p.scale);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                // dimension d belongs to lane c's run: for D 128 c = d / 32 and k step (d % 32) / 4; for 64 runs of 16;
                // for 256 two halves of 128
                const int d = i * 64 + lane * 2;
                constexpr int RUN = D == 64 ? 16 : 32;
                const int half = D == 256 ? d >> 7 : 0, dd = D == 256 ? d & 127 : d;
                const int cc = dd / RUN, ks = half * (RUN / 4) + (dd % RUN) / 4, pair = (dd % 4) / 2;
                uint32_t* f = reinterpret_cast<uint32_t*>(s_q + (r / 8 * (KS / 2) + ks / 2) * 32 + (r % 8) * 4 + cc);
                f[(ks & 1) * 2 + pair] = f16x2_bits(x[2 * i] * down, x[2 * i + 1] * down);
            }
        }
        named_sync(1, C::W * 32);
        uint32_t qf[C::QREG ? NR : 1][C::QREG ? KS : 1][2];
        if constexpr (C::QREG) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < KS / 2; ++i) {
                    const uint4 v = s_q[(n * (KS / 2) + i) * 32 + lane];
                    qf[n][2 * i][0] = v.x, qf[n][2 * i][1] = v.y, qf[n][2 * i + 1][0] = v.z, qf[n][2 * i + 1][1] = v.w;
                }
        }
        // rows 2c and 2c + 1 of each group of 8
        float o[DT][NR][4], m[NR][2], l[NR][2], sc[NR][2];
        int limit[NR][2];  // keys that the row sees
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = n * 8 + 2 * c + h;
                m[n][h] = kNone;
                l[n][h] = 0.f;
                sc[n][h] = s_sc[r];
                limit[n][h] = y.x.kv - y.x.qlen + (y.r0 + r) / p.G + 1;
            }
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
        }
        const int all_see = y.x.kv - y.x.qlen + y.r0 / p.G + 1;  // keys that every row sees

        for (int kt = y.kt0; kt < y.kt1; ++kt, ++it) {
            const uint32_t stage = it % C::STAGES;
            if (!dead && !__all_sync(~0u, mbar_wait_bounded(full + 8 * stage, (it / C::STAGES) & 1, GDN_WAIT_POLLS))) {
                dead = true;
                bits |= GDN_ERRBIT_TIMEOUT;
                s_dead = 1;
            }
            const uint8_t* st = pool + stage * C::STAGE;
            const uint8_t *kc = st, *vc = st + C::TILE * C::CB, *ksc = st + 2 * C::TILE * C::CB, *vsc = ksc + C::TILE * C::SB;
#pragma unroll 1
            for (int step = 0; step < C::STEPS; ++step) {
                const int w0 = (step * C::W + warp) * WT;  // the warp's first token in the tile
                const int tok0 = kt * C::TILE + w0;
                if (tok0 >= y.x.kv || dead) break;
                // S^T: row g of token group j is token j * 8 + (g ^ ((g >> 1) & 1))
                float s[NT / 2][NR][4];
#pragma unroll
                for (int j = 0; j < NT / 2; ++j)
#pragma unroll
                    for (int n = 0; n < NR; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.f;
                constexpr int WN = D == 64 ? 2 : 4;
#pragma unroll
                for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
                    uint32_t w[NT][WN], scl[NT][2];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int r = w0 + j * 8 + (g ^ ((g >> 1) & 1));
                        if constexpr (D == 64) {
                            const uint2 v = *reinterpret_cast<const uint2*>(kc + code_off<D>(r, c >> 1) + (c & 1) * 8);
                            w[j][0] = v.x, w[j][1] = v.y;
                            scl[j][0] = scl[j][1] = e4m3x2_to_f16(ksc[r * 4 + c] * 0x101u);
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(kc + code_off<D>(r, half * 4 + c));
                            w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
                            const uint32_t f =
                                e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(ksc + r * C::SB + half * 8 + c * 2));
                            scl[j][0] = __byte_perm(f, f, 0x1010);
                            scl[j][1] = __byte_perm(f, f, 0x3232);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < WN; ++i) {
                        uint32_t q[NR][4];  // two k steps
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            if constexpr (C::QREG) {
                                const int ks = half * 8 + 2 * i;
                                q[n][0] = qf[n][ks][0], q[n][1] = qf[n][ks][1], q[n][2] = qf[n][ks + 1][0], q[n][3] = qf[n][ks + 1][1];
                            } else {
                                const uint4 v = s_q[(n * (KS / 2) + half * 4 + i) * 32 + lane];
                                q[n][0] = v.x, q[n][1] = v.y, q[n][2] = v.z, q[n][3] = v.w;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < NT / 2; ++j) {
                            uint32_t fa[4], fb[4];
                            e2m1x8_to_f16(w[2 * j][i], fa);
                            e2m1x8_to_f16(w[2 * j + 1][i], fb);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                fa[x] = hmul2(fa[x], scl[2 * j][i / 2]);
                                fb[x] = hmul2(fb[x], scl[2 * j + 1][i / 2]);
                            }
                            const uint32_t a0[4] = {fa[0], fb[0], fa[1], fb[1]}, a1[4] = {fa[2], fb[2], fa[3], fb[3]};
#pragma unroll
                            for (int n = 0; n < NR; ++n) mma_f16(s[j][n], a0, q[n][0], q[n][1]);
#pragma unroll
                            for (int n = 0; n < NR; ++n) mma_f16(s[j][n], a1, q[n][2], q[n][3]);
                        }
                    }
                }
                // softmax in units of log 2; s[j][n]: groups 2j (first two) and 2j + 1, rows 2c and 2c + 1
                bool above = false;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int j = 0; j < NT / 2; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[j][n][i] *= sc[n][i & 1];
                if (tok0 + WT > all_see) {
                    const int tk = tok0 + (g ^ ((g >> 1) & 1));
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int j = 0; j < NT / 2; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (tk + (2 * j + (i >> 1)) * 8 >= limit[n][i & 1]) s[j][n][i] = -INFINITY;
                }
                float top[NR][2];
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = fmaxf(s[0][n][h], s[0][n][2 + h]);
#pragma unroll
                        for (int j = 1; j < NT / 2; ++j) x = fmaxf(x, fmaxf(s[j][n][h], s[j][n][2 + h]));
                        top[n][h] = x;
                        above |= x > m[n][h] + (kSlack + kLift);
                    }
                if (__any_sync(~0u, above)) {
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = top[n][h];
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                            const float mn = fmaxf(m[n][h], x - kLift);
                            const float f = exp2_fast(m[n][h] - mn);
                            m[n][h] = mn;
                            l[n][h] *= f;
#pragma unroll
                            for (int i = 0; i < DT; ++i) {
                                o[i][n][h] *= f;
                                o[i][n][2 + h] *= f;
                            }
                        }
                }
                uint32_t pf[NT][NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float e0 = exp2_fast(s[j >> 1][n][(j & 1) * 2] - m[n][0]), e1 = exp2_fast(s[j >> 1][n][(j & 1) * 2 + 1] - m[n][1]);
                        l[n][0] += e0;
                        l[n][1] += e1;
                        pf[j][n] = movmatrix(f16x2_bits(e0, e1));
                    }
                }
                // O^T += V^T P^T: 16 tokens at a time; this lane's tokens are 2c, 2c + 1 of two groups, swapped for odd c
                const bool tail = tok0 + WT > y.x.kv;  // what lies behind the last token may be anything, NaN scales too
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    constexpr int VN = D / 64;  // words of a run of D / 8 dimensions
                    uint32_t w[4][VN], sv[2][VN > 2 ? 2 : 1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 2 * c + (i & 1), r = w0 + (j + (i >> 1)) * 8 + (n ^ (c & 1));
                        if constexpr (D == 64) {
                            w[i][0] = *reinterpret_cast<const uint32_t*>(vc + code_off<D>(r, g >> 2) + (g & 3) * 4);
                        } else if constexpr (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(vc + code_off<D>(r, g >> 1) + (g & 1) * 8);
                            w[i][0] = v.x, w[i][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(vc + code_off<D>(r, g));
                            w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int ra = w0 + (j + i) * 8 + ((2 * c) ^ (c & 1)), rb = w0 + (j + i) * 8 + ((2 * c + 1) ^ (c & 1));
                        uint32_t x, z;
                        if constexpr (D == 256) {
                            x = *reinterpret_cast<const uint16_t*>(vsc + ra * 16 + g * 2);
                            z = *reinterpret_cast<const uint16_t*>(vsc + rb * 16 + g * 2);
                        } else {
                            const int gr = D == 64 ? g >> 1 : g;
                            x = vsc[ra * C::SB + gr];
                            z = vsc[rb * C::SB + gr];
                        }
                        if (tail) {
                            if (kt * C::TILE + ra >= y.x.kv) x = 0;
                            if (kt * C::TILE + rb >= y.x.kv) z = 0;
                        }
                        if constexpr (D == 256) {
                            sv[i][0] = nan_as_zero(e4m3x2_to_f16(__byte_perm(x, z, 0x0040)));
                            sv[i][1] = nan_as_zero(e4m3x2_to_f16(__byte_perm(x, z, 0x0051)));
                        } else {
                            sv[i][0] = nan_as_zero(e4m3x2_to_f16(x | (z << 8)));
                        }
                    }
#pragma unroll
                    for (int x = 0; x < VN; ++x) {
                        // bytes (token a, token b) of one dimension: even dimensions, then odd ones
                        uint32_t f[2][2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t wa = w[2 * i][x], wb = w[2 * i + 1][x];
                            e2m1x8_to_f16((wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u), f[i][0]);
                            e2m1x8_to_f16(((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u), f[i][1]);
                            const uint32_t sf = sv[i][D == 256 ? x / 2 : 0];
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                f[i][0][z] = hmul2(f[i][0][z], sf);
                                f[i][1][z] = hmul2(f[i][1][z], sf);
                            }
                        }
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint32_t a[4] = {f[0][0][z], f[0][1][z], f[1][0][z], f[1][1][z]};
#pragma unroll
                            for (int n = 0; n < NR; ++n) mma_f16(o[x * 4 + z][n], a, pf[j][n], pf[j + 1][n]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(empty + 8 * stage);  // (a stage whose copy never came is not filled again)
        }

        // ---- the warps' parts of the item joined, a group of rows of each warp at a time, and stored ---------------
        const bool whole = y.kt0 == 0 && y.kt1 == y.kts;
        float* part = parts + ((int64_t)blockIdx.x * 2 + (y.kt0 == 0 ? 1 : 0)) * part_floats(C::ROWS, D);
        constexpr int RC = D / 32, CH = D / 4;  // 16-byte chunks of a run and of a row
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            named_sync(1, C::W * 32);  // the rows before are read (and s_sc, the fragments of Q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = l[n][h];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                if (g == 0) s_ml[warp * 8 + 2 * c + h] = make_float2(m[n][h], x);
                // runs' chunks XORed with their lane so that the stores of different lanes meet few banks twice
                float* dst = s_o + (warp * 8 + 2 * c + h) * C::OROW + g * (D / 8);
#pragma unroll
                for (int i = 0; i < RC; ++i)
                    *reinterpret_cast<float4*>(dst + ((i ^ (g & (RC < 4 ? RC - 1 : 3))) << 2)) =
                        make_float4(o[2 * i][n][h], o[2 * i][n][2 + h], o[2 * i + 1][n][h], o[2 * i + 1][n][2 + h]);
            }
            named_sync(1, C::W * 32);
            if (s_dead) continue;
            for (int idx = tid; idx < 8 * CH; idx += C::W * 32) {
                const int rr = idx / CH, ch = idx % CH, r = n * 8 + rr;
                if (r >= nrows) continue;
                float mm = -INFINITY, ll = 0.f;
#pragma unroll
                for (int w = 0; w < C::W; ++w) mm = fmaxf(mm, s_ml[w * 8 + rr].x);
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                const int gg = ch / RC, j = ch % RC, at = gg * (D / 8) + ((j ^ (gg & (RC < 4 ? RC - 1 : 3))) << 2);
#pragma unroll
                for (int w = 0; w < C::W; ++w) {
                    const float2 x = s_ml[w * 8 + rr];
                    const float f = mm == -INFINITY ? 1.f : exp2_fast(x.x - mm);
                    ll += x.y * f;
                    const float4 v = *reinterpret_cast<const float4*>(s_o + (w * 8 + rr) * C::OROW + at);
                    a.x = fmaf(v.x, f, a.x);
                    a.y = fmaf(v.y, f, a.y);
                    a.z = fmaf(v.z, f, a.z);
                    a.w = fmaf(v.w, f, a.w);
                }
                if (whole) {
                    const int t = (y.r0 + r) / p.G, h = y.hk * p.G + (y.r0 + r) - t * p.G;
                    const int64_t out = (int64_t)(y.x.q0 + t) * p.HQ + h;
                    const float inv = ll > 0.f ? p.kv.v_scale / ll : ll != ll ? ll : 0.f;
                    *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + out * D + ch * 4) =
                        make_uint2(bf16x2_bits(a.x * inv, a.y * inv), bf16x2_bits(a.z * inv, a.w * inv));
                    if (p.lse && ch == 0) p.lse[out] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
                } else {
                    *reinterpret_cast<float4*>(part + (int64_t)r * D + ch * 4) = a;
                    if (ch == 0) *reinterpret_cast<float2*>(part + (int64_t)C::ROWS * D + 2 * r) = make_float2(mm, ll);
                }
            }
        }
        if (!whole && y.kt0 == 0 && tid == 0 && !s_dead) {
            desc->last = cta_of(all, ctas, walk.u - (y.kt1 - y.kt0) + y.kts - 1);
            desc->rows = nrows;
            desc->q0 = y.x.q0;
            desc->r0 = y.r0;
            desc->hk = y.hk;
        }
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);
}

// Joins the parts of items that more than one CTA worked on: block (x, y) takes rows y, y + gridDim.y, .. of the item that
// CTA x began and did not end.  Few parts: a warp takes a row.  Many: the block takes a row, D / 4 threads a part of it, and
// as many parts side by side as that leaves room for.  Latency bound: 5.6 us for a decode's parts (12.5 us for 256 rows of D 128
// from every CTA, 25 MB), of which the programmatic launch hides the start.
constexpr int kJoinThreads = 128;
constexpr int kFewParts = 4;
constexpr int kMaxParts = 1024;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 8) gdn_kv4_attention_join_kernel(Kv4AttentionParams p, int rows_max, int ctas) {
    __shared__ float s_f[kMaxParts];
    __shared__ float s_red[2 * kJoinThreads / 32];
    __shared__ float4 s_acc[kJoinThreads];
    grid_dependency_wait();
    const PartDesc d = reinterpret_cast<const PartDesc*>(p.workspace)[blockIdx.x];
    if (d.last < 0) return;
    const float* parts = reinterpret_cast<const float*>(reinterpret_cast<const PartDesc*>(p.workspace) + ctas);
    const int first = blockIdx.x, n = d.last - first + 1, tid = threadIdx.x;
    const int64_t step = part_floats(rows_max, D);
    auto part = [&](int i) { return parts + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * step; };
    auto store = [&](int r, int ch, float4 a, float mm, float ll) {
        const int t = (d.r0 + r) / p.G, h = d.hk * p.G + (d.r0 + r) - t * p.G;
        const int64_t out = (int64_t)(d.q0 + t) * p.HQ + h;
        const float inv = ll > 0.f ? p.kv.v_scale / ll : ll != ll ? ll : 0.f;
        *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + out * D + ch * 4) =
            make_uint2(bf16x2_bits(a.x * inv, a.y * inv), bf16x2_bits(a.z * inv, a.w * inv));
        if (ch == 0 && p.lse) p.lse[out] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
    };
    if (n <= kFewParts) {  // a row a warp: nothing to exchange, all loads at once
        const int lane = tid & 31;
        constexpr int V = (D / 4 + 31) / 32;
        for (int r = blockIdx.y * (kJoinThreads / 32) + (tid >> 5); r < d.rows; r += gridDim.y * (kJoinThreads / 32)) {
            float2 ml[kFewParts];
            float4 v[kFewParts][V];
#pragma unroll
            for (int i = 0; i < kFewParts; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                if (i >= n) continue;
                ml[i] = *reinterpret_cast<const float2*>(part(i) + (int64_t)rows_max * D + 2 * r);
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (lane + 32 * k < D / 4) v[i][k] = *reinterpret_cast<const float4*>(part(i) + (int64_t)r * D + (lane + 32 * k) * 4);
            }
            float mm = ml[0].x, ll = 0.f;
#pragma unroll
            for (int i = 1; i < kFewParts; ++i) mm = fmaxf(mm, ml[i].x);
            float4 a[V];
#pragma unroll
            for (int k = 0; k < V; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kFewParts; ++i) {
                if (i >= n) continue;
                const float f = mm == -INFINITY ? 1.f : exp2_fast(ml[i].x - mm);
                ll = fmaf(ml[i].y, f, ll);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    a[k].x = fmaf(v[i][k].x, f, a[k].x);
                    a[k].y = fmaf(v[i][k].y, f, a[k].y);
                    a[k].z = fmaf(v[i][k].z, f, a[k].z);
                    a[k].w = fmaf(v[i][k].w, f, a[k].w);
                }
            }
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (lane + 32 * k < D / 4) store(r, lane + 32 * k, a[k], mm, ll);
        }
        return;
    }
    for (int r = blockIdx.y; r < d.rows; r += gridDim.y) {
        float mm = -INFINITY;
        for (int i = tid; i < n; i += kJoinThreads) mm = fmaxf(mm, part(i)[(int64_t)rows_max * D + 2 * r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
        if ((tid & 31) == 0) s_red[tid >> 5] = mm;
        __syncthreads();
        mm = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
        float ll = 0.f;
        for (int i = tid; i < n; i += kJoinThreads) {
            const float2 x = *reinterpret_cast<const float2*>(part(i) + (int64_t)rows_max * D + 2 * r);
            const float f = mm == -INFINITY ? 1.f : exp2_fast(x.x - mm);
            s_f[i] = f;
            ll = fmaf(x.y, f, ll);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(~0u, ll, o);
        if ((tid & 31) == 0) s_red[4 + (tid >> 5)] = ll;
        __syncthreads();
        ll = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
        constexpr int TR = D / 4, GR = kJoinThreads / TR;  // threads of a row; parts side by side
        const int ch = tid % TR, gr = tid / TR;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = gr; i < n; i += GR) {
            const float4 v = *reinterpret_cast<const float4*>(part(i) + (int64_t)r * D + ch * 4);
            const float f = s_f[i];
            a.x = fmaf(v.x, f, a.x);
            a.y = fmaf(v.y, f, a.y);
            a.z = fmaf(v.z, f, a.z);
            a.w = fmaf(v.w, f, a.w);
        }
        s_acc[tid] = a;
        __syncthreads();
        if (gr == 0) {
#pragma unroll
            for (int k = 1; k < GR; ++k) {
                const float4 v = s_acc[k * TR + ch];
                a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
            }
            store(r, ch, a, mm, ll);
        }
        __syncthreads();
    }
}

constexpr int kCtasPerSm = 2;  // at most
static_assert(kCtasPerSm * 200 <= kMaxParts, "parts of an item");

// CTAs of an SM, found once for each kernel and device
template <typename C>
cudaError_t resident(int* n) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaFuncSetAttribute(gdn_kv4_attention_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, gdn_kv4_attention_kernel<C>, C::THREADS, C::SMEM);
    if (e != cudaSuccess) return e;
    // the warps' registers are split anew in the kernel: the block has to hold what that sums up to
    cudaFuncAttributes at{};
    e = cudaFuncGetAttributes(&at, gdn_kv4_attention_kernel<C>);
    if (e != cudaSuccess) return e;
    if (at.numRegs != C::LREG) return cudaErrorLaunchOutOfResources;
    *n = *n < 1 ? 1 : *n > kCtasPerSm ? kCtasPerSm : *n;
    if (dev < 64) known[dev].store(*n, std::memory_order_relaxed);
    return cudaSuccess;
}

template <typename C>
cudaError_t run(const Kv4AttentionParams& p, cudaStream_t s) {
    const int sms = sm_count();
    if (sms == 0) return cudaErrorNoDevice;
    int per = 0;
    CUtensorMap map;
    cudaError_t e = resident<C>(&per);
    if (e == cudaSuccess) e = codes_map(p.kv, C::TILE, &map);
    if (e != cudaSuccess) return e;
    const int ctas = sms * per;
    gdn_kv4_attention_kernel<C><<<ctas, C::THREADS, C::SMEM, s>>>(p, map);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_kv4_join(p, C::ROWS, ctas, s);
}

// More rows than this go to the tcgen05 kernel, although 128 is what it wants: 256 lanes of 64 rows over 2100 keys, D 64, took
// 255 us there and 352 us here (160 us there now).  17 to 32 rows stay here; there and here, 128 lanes over up to 16384 keys: 32 rows of
// D 64 254 and 244 us, of D 128 391 and 307, of D 256 396 and 319; 20 rows of D 64 246 and 225, of D 256 382 and 307.
bool wide(int64_t rows) { return rows > 32; }

// Rows of an item: 8, 16 or 32; of D 256 at most 16 (O^T takes D * rows / 32 registers a thread), more take several items
int item_rows(int64_t rows, int D) { return rows <= 8 ? 8 : rows <= 16 || D == 256 ? 16 : 32; }

template <int D>
cudaError_t run_join(const Kv4AttentionParams& p, int rows, int ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, rows <= 64 ? 8 : rows / 16);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_kv4_attention_join_kernel<D>, p, rows, ctas);
}

}  // namespace

cudaError_t launch_kv4_join(const Kv4AttentionParams& p, int rows, int ctas, cudaStream_t s) {
    return p.kv.D == 64    ? run_join<64>(p, rows, ctas, s)
           : p.kv.D == 128 ? run_join<128>(p, rows, ctas, s)
                           : run_join<256>(p, rows, ctas, s);
}

cudaError_t launch_kv4_attention(const Kv4AttentionParams& p, cudaStream_t s) {
    if (wide((int64_t)p.T * p.G)) return launch_kv4_attention_wide(p, s);
    const int rows = item_rows((int64_t)p.T * p.G, p.kv.D);
    switch (p.kv.D * 100 + rows) {
    case 6408: return run<Cfg<64, 1, 32, 256, 3, 2, 0>>(p, s);
    case 6416: return run<Cfg<64, 2, 32, 256, 3, 2, 1>>(p, s);
    case 6432: return run<Cfg<64, 4, 16, 128, 4, 1, 3>>(p, s);
    case 12808: return run<Cfg<128, 1, 32, 256, 2, 2, 2>>(p, s);
    case 12816: return run<Cfg<128, 2, 32, 256, 4, 1, 3>>(p, s);
    case 12832: return run<Cfg<128, 4, 16, 128, 4, 1, 6>>(p, s);
    case 25608: return run<Cfg<256, 1, 16, 128, 3, 1, 3>>(p, s);
    default: return run<Cfg<256, 2, 16, 128, 3, 1, 5>>(p, s);
    }
}

int64_t kv4_attention_workspace(int B, int T, int HQ, int HK, int D) {
    (void)B;
    // a call may bring fewer rows than this: the most that any kernel up to them wants
    const int64_t rows = (int64_t)T * (HQ / HK);
    const int sms = sm_count();
    const int64_t ctas = (int64_t)(sms > 0 ? sms : 152) * kCtasPerSm;
    const int64_t n = ctas * ((int64_t)sizeof(PartDesc) + 2 * part_floats(item_rows(rows, D), D) * 4);
    return wide(rows) ? std::max(n, kv4_attention_wide_workspace(D)) : n;
}

}  // namespace gdn
