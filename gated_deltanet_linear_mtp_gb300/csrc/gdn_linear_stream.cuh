// gdn_linear_stream.cuh -- steps of many lanes: linear attention with states that a persistent kernel streams through shared
// memory (included by gdn_linear.cuh, whose formulas, products and lane layout it shares).
//
// A state is one run of bytes, so a tile of 64 or 128 of its rows is one bulk copy.  A CTA walks tiles; one warp asks for the state and
// the tokens' q, k, v of up to four tiles ahead, as many as fit (the slots of 32 tiles at once), a second forms what all rows share
// (w_tj, and whether k is finite), and the others take 16 rows each.  Thus 64 to 128 KB an SM stay in flight whatever the
// products wait for, which a CTA per tile does not reach: its loads stand behind its slot, and its stores behind its products.
//   * The update sum_j (g^(n-1-j) v_j) k_j^T is a product as well: A = v_j g^(n-1-j) in three bf16 parts, two of them side by side as
//     the 16 columns of one instruction; B = k transposed by its load.  k's words lie permuted in shared memory so that a lane's sums are of
//     the eight columns of S that it holds.  Values that are not finite take the sum term by term.
// Measured in graph replays (HK 16, HV 32, D 128, bf16 states): verify of 256 lanes x 8 tokens 49.2 us (6.5 TB/s; a CTA per 64 rows 66.8),
// their commit 91 in place, 96 into other slots (6 and 5.7 TB/s of mixed traffic; 110 in place), decode of 256 lanes 89 and 94 (96 in place);
// verify of 128 lanes x 8 with fp32 states 47.5 (6.2 TB/s; 56).  Writing the states by bulk copies from shared memory measured the same (88.7 against 88.2).
#pragma once

#include "gdn_tcgen05.cuh"

namespace gdn {

constexpr int kLsTokens = 8;       // tokens of a step at most
constexpr int kLsSmem = 113 * 1024;  // of a CTA: two fit an SM

template <int DK, typename StT, int kMode>
struct LinStream {
    static constexpr bool OUT = kMode != kLinCommit, UPDATE = kMode != kLinVerify;
    static_assert(!UPDATE || sizeof(StT) == 2, "fp32 states are only read here");
    static constexpr int W = DK * sizeof(StT) <= 256 ? 8 : 4;  // warps with 16 rows each
    static constexpr int ROWS = 16 * W, THREADS = 32 * (W + 2);  // and one that loads, one for what all rows share
    static constexpr int STATE = ROWS * DK * (int)sizeof(StT);
    // Bytes from token to token.  Two rows of 64 bytes (q, k) fall into different banks, and so do eight of 16 (k to be transposed)
    // and the words that a warp takes of four pairs of tokens of v.
    static constexpr int QP = 2 * DK + 64, KP = UPDATE ? 2 * DK + 16 : QP, VP = 2 * ROWS + 16;
    static constexpr int Q0 = STATE, K0 = Q0 + (OUT ? kLsTokens * QP : 0), V0 = K0 + kLsTokens * KP, W0 = V0 + kLsTokens * VP,
                         D0 = W0 + (OUT ? 4 * kLsTokens * kLsTokens : 0), BYTES = D0 + 32;
    static constexpr int FIT = (kLsSmem - 256) / BYTES, NS = FIT < 4 ? FIT : 4;
    static constexpr int SMEM = NS * BYTES + 24 * NS + 16;
    static_assert(NS >= 2 && BYTES % 16 == 0 && SMEM <= kLsSmem, "two CTAs of two stages fit an SM");
};

__device__ __forceinline__ void cp_async_or_zero16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_or_zero4(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
// one arrival at `bar` once this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// four 8 x 8 matrices, transposed: two rows' elements of one column a register
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// the product of 8 columns of A
__device__ __forceinline__ void mma_bf16_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ bool pair_not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int DK, typename StT, int kMode>
__global__ void __launch_bounds__(LinStream<DK, StT, kMode>::THREADS, 2)
    gdn_linear_stream_kernel(const LinearParams p, const uint32_t tiles) {
    using L = LinStream<DK, StT, kMode>;
    using bf16 = __nv_bfloat16;
    constexpr int NP = DK / 32, NS = L::NS, W = L::W;
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t base = smem_u32(smem), bars = base + NS * L::BYTES;
    volatile int* const fail = reinterpret_cast<volatile int*>(smem + NS * L::BYTES + 24 * NS);
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (NS + s); };
    auto ready = [&](int s) { return bars + 8 * (2 * NS + s); };
    // of a whole warp, bounded: a wait that runs out ends the CTA's work.  Every branch goes by a vote, so that the warp stays together for its
    // products and transposed loads.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
        for (uint32_t i = 0; !ok && i < GDN_WAIT_POLLS && !__any_sync(0xffffffffu, *fail != 0); ++i)
            ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
        return ok;
    };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3, T = p.T;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 33);  // the state's copy, and the loading warp's lanes
            mbar_init(empty(s), W + 1);
            mbar_init(ready(s), 1);
        }
        *fail = 0;
        fence_mbar_init();
    }
    for (int s = 0; s < NS; ++s)  // tokens behind the last stay zero
        for (int e = tid; e < (L::W0 - L::Q0) / 16; e += L::THREADS)
            reinterpret_cast<uint4*>(smem + s * L::BYTES + L::Q0)[e] = make_uint4(0, 0, 0, 0);
    __syncthreads();

    if (warp == W) {  // ---- loads ----
        const uint32_t nrb = (uint32_t)(p.DV + L::ROWS - 1) / L::ROWS, G = gridDim.x;
        const int R = p.HV / p.HK;
        uint32_t used = 0;
        bool ok = true;
        for (uint64_t first = blockIdx.x; first < tiles && ok; first += 32ull * G) {
            const uint64_t t = first + (uint64_t)lane * G;  // a tile a lane: its slots are asked for at once
            int b = 0, h = 0, row0 = 0, slot = -1, out = -1, n = T;
            float ld = 0.f;
            if (t < tiles) {
                const uint32_t bh = (uint32_t)t / nrb;
                row0 = (int)((uint32_t)t - bh * nrb) * L::ROWS;
                b = (int)(bh / (uint32_t)p.HV);
                h = (int)(bh - (uint32_t)b * (uint32_t)p.HV);
                slot = p.indices[b];
                if (L::UPDATE) out = p.out_indices != nullptr ? p.out_indices[b] : slot;
                if (kMode == kLinCommit) n = p.steps[b];
                ld = p.log_decay[h];
            }
            bool take = slot != -1;
            if (take && (slot < -1 || slot >= p.num_slots || out < -1 || out >= p.num_slots)) {
                if (p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
                take = false;
            }
            if (kMode == kLinCommit && take) {
                if (n < 0 || n > T) {
                    if (p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_ACCEPT_LEN);
                    take = false;
                } else if (out < 0 || (n == 0 && out == slot)) {
                    take = false;  // nothing to write
                }
            }
            for (uint32_t todo = __ballot_sync(0xffffffffu, take); todo != 0; todo &= todo - 1) {
                const int src = __ffs(todo) - 1;
                const int tb = __shfl_sync(0xffffffffu, b, src), th = __shfl_sync(0xffffffffu, h, src),
                          tr = __shfl_sync(0xffffffffu, row0, src), tn = __shfl_sync(0xffffffffu, n, src),
                          ts = __shfl_sync(0xffffffffu, slot, src), to = __shfl_sync(0xffffffffu, out, src);
                const float tl = __shfl_sync(0xffffffffu, ld, src);
                const int s = (int)(used % NS);
                if (used >= NS && !wait(empty(s), (used / NS - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t st = base + s * L::BYTES;
                if (lane == 0) {
                    int* d = reinterpret_cast<int*>(smem + s * L::BYTES + L::D0);
                    d[0] = tb, d[1] = th, d[2] = tr, d[3] = to, d[4] = tn, d[5] = __float_as_int(tl), d[6] = 0;
                    const uint32_t bytes = (uint32_t)min(L::ROWS, p.DV - tr) * DK * (uint32_t)sizeof(StT);
                    mbar_arrive_expect_tx(full(s), bytes);
                    const StT* from = static_cast<const StT*>(p.pool) + (((int64_t)ts * p.HV + th) * p.DV + tr) * DK;
#ifdef GDN_TEST_MISSING_COPY
                    if (blockIdx.x != 0 || used != 0)
#endif
                        bulk_g2s(st, from, bytes, full(s));
                }
                const int64_t tok = (int64_t)tb * T;
                const bf16* kp = static_cast<const bf16*>(p.k) + (tok * p.HK + th / R) * DK;
                const bf16* vp = static_cast<const bf16*>(p.v) + (tok * p.HV + th) * p.DV + tr;
                const int64_t kstep = (int64_t)p.HK * DK, vstep = (int64_t)p.HV * p.DV;
                if constexpr (L::UPDATE) {
#pragma unroll 4
                    for (int e = lane; e < T * (DK / 2); e += 32) {  // word 16 c + 4 t + i goes to 16 c + 4 i + t
                        const int j = e / (DK / 2), x = e % (DK / 2);
                        cp_async_or_zero4(st + L::K0 + j * L::KP + 4 * ((x & ~15) + 4 * (x & 3) + ((x >> 2) & 3)),
                                          kp + j * kstep + 2 * x, j < tn);
                    }
                } else {
#pragma unroll 4
                    for (int e = lane; e < T * (DK / 8); e += 32) {
                        const int j = e / (DK / 8), x = e % (DK / 8);
                        cp_async_or_zero16(st + L::K0 + j * L::KP + 16 * x, kp + j * kstep + 8 * x, j < tn);
                    }
                }
                if constexpr (L::OUT) {
                    const bf16* qp = static_cast<const bf16*>(p.q) + (tok * p.HK + th / R) * DK;
#pragma unroll 4
                    for (int e = lane; e < T * (DK / 8); e += 32) {
                        const int j = e / (DK / 8), x = e % (DK / 8);
                        cp_async_or_zero16(st + L::Q0 + j * L::QP + 16 * x, qp + j * kstep + 8 * x, true);
                    }
                }
#pragma unroll 4
                for (int e = lane; e < T * (L::ROWS / 8); e += 32) {
                    const int j = e / (L::ROWS / 8), x = e % (L::ROWS / 8);
                    const bool real = j < tn && tr + 8 * x < p.DV;
                    cp_async_or_zero16(st + L::V0 + j * L::VP + 16 * x, vp + j * vstep + (real ? 8 * x : 0), real);
                }
                cp_async_arrive(full(s));
                ++used;
            }
        }
        if (ok) {  // the mark of the end
            const int s = (int)(used % NS);
            if (used >= NS && !wait(empty(s), (used / NS - 1) & 1)) {
                ok = false;
            } else {
                if (lane == 0) {
                    *reinterpret_cast<int*>(smem + s * L::BYTES + L::D0) = -1;
                    mbar_arrive(full(s));
                }
                cp_async_arrive(full(s));
            }
        }
        // the CTA leaves when its copies have landed, also where a wait ran out (the mark has taken the stage of `used - NS`)
        if (!ok) *fail = 1;
        for (uint32_t u = used < (uint32_t)NS ? 0 : used - NS + ok; u < used; ++u)
            mbar_wait_bounded(full((int)(u % NS)), (u / NS) & 1, GDN_WAIT_POLLS);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        for (uint32_t it = 0;; ++it) {
            const int s = (int)(it % NS);
            const uint32_t parity = (it / NS) & 1;
            if (!wait(full(s), parity)) {
                *fail = 1;
                break;
            }
            unsigned char* const st = smem + s * L::BYTES;
            int* const d = reinterpret_cast<int*>(st + L::D0);
            const int b = d[0], h = d[1], out = d[3], n = d[4];
            if (b < 0) break;
            const float pw = decay_power(__int_as_float(d[5]), lane);  // lane e: g^e (up to 8)
            auto power = [&](int e) { return __shfl_sync(0xffffffffu, pw, e & 31); };

            if (warp > W) {  // ---- w_tj = g^(t-j) (k_j . q_t), and whether k is finite ----
                float w[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                bool odd = false;
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    uint4 kf;
                    if constexpr (L::UPDATE) {
                        const uint32_t* kr = reinterpret_cast<const uint32_t*>(st + L::K0 + g * L::KP) + 16 * c + t4;
                        kf = make_uint4(kr[0], kr[4], kr[8], kr[12]);
                        odd |= pair_not_finite(kf.x) || pair_not_finite(kf.y) || pair_not_finite(kf.z) || pair_not_finite(kf.w);
                    } else {
                        kf = *reinterpret_cast<const uint4*>(st + L::K0 + g * L::KP + 64 * c + 16 * t4);
                    }
                    if constexpr (L::OUT) {
                        const uint4 qf = *reinterpret_cast<const uint4*>(st + L::Q0 + g * L::QP + 64 * c + 16 * t4);
                        mma_bf16(w[0], qf.x, 0u, qf.y, 0u, kf.x, kf.y);
                        mma_bf16(w[1], qf.z, 0u, qf.w, 0u, kf.z, kf.w);
                    }
                }
                if constexpr (L::OUT) {
                    float2 x;
                    const int j = 2 * t4;
                    const float f0 = power(g - j), f1 = power(g - j - 1);
                    x.x = j <= g ? f0 * (w[0][0] + w[1][0]) : 0.f;
                    x.y = j + 1 <= g ? f1 * (w[0][1] + w[1][1]) : 0.f;
                    reinterpret_cast<float2*>(st + L::W0)[lane] = x;
                }
                if constexpr (L::UPDATE) {
                    odd = __any_sync(0xffffffffu, odd);
                    if (lane == 0) d[6] = odd;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ready(s));
                    mbar_arrive(empty(s));
                }
                continue;
            }

            const int lrow = 16 * warp + 2 * g, row = d[2] + lrow;  // and the next
            const bool live = row < p.DV;
            RowPiece<StT> S[2][NP];
            {
                const bool o = g & 1;  // lanes of odd g take the other half first: all banks serve
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const unsigned char* src = st + (lrow + r) * DK * (int)sizeof(StT);
                    if constexpr (sizeof(StT) == 4) {
#pragma unroll
                        for (int c = 0; c < NP; ++c) {
                            const float4 x = *reinterpret_cast<const float4*>(src + 128 * c + 32 * t4 + 16 * o);
                            const float4 y = *reinterpret_cast<const float4*>(src + 128 * c + 32 * t4 + 16 * !o);
                            S[r][c].a = o ? y : x;
                            S[r][c].b = o ? x : y;
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < NP; c += 2) {
                            const uint4 x = *reinterpret_cast<const uint4*>(src + 64 * (c + o) + 16 * t4);
                            const uint4 y = *reinterpret_cast<const uint4*>(src + 64 * (c + !o) + 16 * t4);
                            S[r][c].r = o ? y : x;
                            S[r][c + 1].r = o ? x : y;
                        }
                    }
                }
            }
            // v of rows row, row + 1: of tokens 2 t4 and 2 t4 + 1
            const uint32_t* vw = reinterpret_cast<const uint32_t*>(st + L::V0) + lrow / 2;
            const uint32_t v0 = vw[2 * t4 * (L::VP / 4)], v1 = vw[(2 * t4 + 1) * (L::VP / 4)];
            const bool odd = __any_sync(0xffffffffu, pair_not_finite(v0) || pair_not_finite(v1));
            const uint32_t va = __byte_perm(v0, v1, 0x5410), vb = __byte_perm(v0, v1, 0x7632);  // row, row + 1
            if constexpr (L::OUT) {
                float dot[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    const uint4 qf = *reinterpret_cast<const uint4*>(st + L::Q0 + g * L::QP + 64 * c + 16 * t4);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        constexpr int NW = RowPiece<StT>::PARTS;
                        uint32_t a0[NW], a1[NW], a2[NW], a3[NW];
                        S[0][c].words(e, a0, a2);
                        S[1][c].words(e, a1, a3);
#pragma unroll
                        for (int i = 0; i < NW; ++i)
                            mma_bf16(dot[e], a0[i], a1[i], a2[i], a3[i], word_of(qf, 2 * e), word_of(qf, 2 * e + 1));
                    }
                }
                if (!wait(ready(s), parity)) {
                    *fail = 1;
                    break;
                }
                float sum[4] = {0.f, 0.f, 0.f, 0.f};  // of rows row (0, 1) and row + 1 (2, 3), tokens 2 t4 and 2 t4 + 1
                if (!odd) {
                    const float2 w = reinterpret_cast<const float2*>(st + L::W0)[lane];
                    uint32_t parts[3];
                    three_parts(w.x, w.y, parts);
                    mma_bf16(sum, va, vb, va, vb, parts[0], parts[1]);
                    mma_bf16_half(sum, va, vb, parts[2]);
                } else {
                    for (int j = 0; j < n; ++j) {
                        const uint32_t x = vw[j * (L::VP / 4)];
                        const float x0 = __uint_as_float(x << 16), x1 = __uint_as_float(x & 0xffff0000u);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float w = reinterpret_cast<const float*>(st + L::W0)[(2 * t4 + e) * kLsTokens + j];
                            if (j <= 2 * t4 + e) {
                                sum[e] = fmaf(w, x0, sum[e]);
                                sum[2 + e] = fmaf(w, x1, sum[2 + e]);
                            }
                        }
                    }
                }
                if constexpr (!L::UPDATE) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty(s));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * t4 + e;
                    const float f = power(t + 1);
                    const float x = p.scale * fmaf(f, dot[0][e] + dot[1][e], sum[e]);
                    const float y = p.scale * fmaf(f, dot[0][2 + e] + dot[1][2 + e], sum[2 + e]);
                    if (t >= T || !live) continue;
                    const int64_t at = (((int64_t)b * T + t) * p.HV + h) * p.DV + row;
                    if (p.out_bf16) {
                        bf16* dst = static_cast<bf16*>(p.o) + at;
                        if (p.o_pair) {
                            *reinterpret_cast<uint32_t*>(dst) = Chunk<bf16>::pack2(x, y);
                        } else {
                            dst[0] = __float2bfloat16_rn(x);
                            dst[1] = __float2bfloat16_rn(y);
                        }
                    } else {
                        float* dst = static_cast<float*>(p.o) + at;
                        dst[0] = x;
                        dst[1] = y;
                    }
                }
            }
            if constexpr (L::UPDATE) {
                if (!L::OUT && !wait(ready(s), parity)) {
                    *fail = 1;
                    break;
                }
                if (out >= 0) {
                    // v_j g^(n-1-j) of rows row and row + 1 in three parts
                    const bool products = n > 0 && !odd && d[6] == 0;  // of no tokens: the state as it is
                    const int e = n - 1 - 2 * t4;
                    float f0 = power(e), f1 = power(e - 1);
                    f0 = e >= 0 ? f0 : 0.f;
                    f1 = e >= 1 ? f1 : 0.f;
                    uint32_t pa[3], pb[3];
                    three_parts(f0 * __uint_as_float(va << 16), f1 * __uint_as_float(va & 0xffff0000u), pa);
                    three_parts(f0 * __uint_as_float(vb << 16), f1 * __uint_as_float(vb & 0xffff0000u), pb);
                    const float2 gn = make_float2(power(n), power(n));
                    bf16* dst = static_cast<bf16*>(p.pool) + (((int64_t)out * p.HV + h) * p.DV + row) * DK + 8 * t4;
#pragma unroll
                    for (int c = 0; c < NP; ++c) {
                        float2 x[2][4];
                        S[0][c].unpack(x[0]);
                        S[1][c].unpack(x[1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[0][i] = __fmul2_rn(gn, x[0][i]);
                            x[1][i] = __fmul2_rn(gn, x[1][i]);
                        }
                        if (products) {
                            // column n of product i is column 32 c + 8 (n / 2) + 2 i + n % 2 of the state: the lane's own
                            uint32_t kc[4];
                            load_transposed(kc, smem_u32(st) + L::K0 + (lane & 7) * L::KP + 64 * c + 16 * (lane >> 3));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float a[4] = {x[0][i].x, x[0][i].y, x[1][i].x, x[1][i].y};
                                mma_bf16(a, pa[0], pb[0], pa[1], pb[1], kc[i], kc[i]);
                                mma_bf16_half(a, pa[2], pb[2], kc[i]);
                                x[0][i] = make_float2(a[0], a[1]);
                                x[1][i] = make_float2(a[2], a[3]);
                            }
                        } else {
                            for (int j = 0; j < n; ++j) {
                                const uint32_t* kr = reinterpret_cast<const uint32_t*>(st + L::K0 + j * L::KP) + 16 * c + t4;
                                const uint4 k1[1] = {make_uint4(kr[0], kr[4], kr[8], kr[12])};
                                float2 k2[4];
                                Slice8<bf16>::unpack(k1, k2);
                                const uint32_t v2 = vw[j * (L::VP / 4)];
                                const float f = power(n - 1 - j);
                                const float y0 = f * __uint_as_float(v2 << 16), y1 = f * __uint_as_float(v2 & 0xffff0000u);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    x[0][i] = __ffma2_rn(make_float2(y0, y0), k2[i], x[0][i]);
                                    x[1][i] = __ffma2_rn(make_float2(y1, y1), k2[i], x[1][i]);
                                }
                            }
                        }
                        if (live) {
                            Slice8<bf16>::store_global<false>(dst + 32 * c, x[0]);
                            Slice8<bf16>::store_global<false>(dst + DK + 32 * c, x[1]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(s));
            }
        }
    }
    __syncthreads();
    if (tid == 0 && *fail != 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_TIMEOUT);
}

template <int DK, typename StT, int kMode>
cudaError_t launch_linear_stream(const LinearParams& p, uint32_t tiles, int sms, cudaStream_t s) {
    using L = LinStream<DK, StT, kMode>;
    auto kernel = gdn_linear_stream_kernel<DK, StT, kMode>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const uint32_t most = 2u * (uint32_t)sms;
    kernel<<<tiles < most ? tiles : most, L::THREADS, L::SMEM, s>>>(p, tiles);
    return cudaGetLastError();
}

// Whether the call is the streaming kernel's; false (nothing launched) otherwise.  It takes what it is faster at, where a tile is
// not half empty and the CTAs get two of them, four an SM (us in graph replays, streaming / a CTA per 64 rows; HV 32, DV 128, bf16 states, DK
// 128): verify of 8 tokens 16 lanes (3.4 tiles an SM) 6.6 / 7.1, 20 lanes 7.8 / 7.9, 32 8.8 / 11.2, 128 27.1 / 35.8, of 4 tokens 20 lanes
// 7.8 / 7.2, 32 9.1 / 9.5, 128 25.3 / 28.8; commit of 20 lanes 10.5 / 11.5; decode of one token 20 lanes 11.3 / 10.8, 32 14.2 / 15.5, 256
// 88.8 / 96.0.  DK 64, 32 lanes: verify 7.4 / 8.4, with fp32 states 9.7 / 11.6.  DV 64 of DK 128, tiles half empty: commit of 64 lanes 16.9 / 16.7,
// decode 18.4 / 15.6.  fp32 states that are written leave no room for either: decode of 64 lanes, DK 128, 47.0 / 45.6.
template <int DK, typename StT>
bool try_linear_stream(const LinearParams& p, cudaStream_t s, cudaError_t& err) {
    if constexpr (DK >= 64) {
        constexpr int ROWS = LinStream<DK, StT, kLinVerify>::ROWS;
        const int64_t blocks = ((int64_t)p.DV + ROWS - 1) / ROWS, tiles = (int64_t)p.B * p.HV * blocks;
        if (p.T > kLsTokens || p.cache != nullptr || !p.v_vec || blocks * ROWS >= 2 * (int64_t)p.DV || tiles > 0x7fffffff ||
            (sizeof(StT) == 4 && p.write))
            return false;
        const int sms = sm_count();
        if (sms == 0 || tiles < 4 * (int64_t)sms) return false;
        if constexpr (sizeof(StT) == 2) {
            if (p.write) {
                err = p.q == nullptr ? launch_linear_stream<DK, StT, kLinCommit>(p, (uint32_t)tiles, sms, s)
                                     : launch_linear_stream<DK, StT, kLinDecode>(p, (uint32_t)tiles, sms, s);
                return true;
            }
        }
        err = launch_linear_stream<DK, StT, kLinVerify>(p, (uint32_t)tiles, sms, s);
        return true;
    } else {
        return false;
    }
}

}  // namespace gdn
