// gdn_linear_prefill.cu -- prompts through linear attention with a fixed decay for each head, on the tensor cores (sm_103a):
//     S_t = g S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
// in chunks of C = 128 tokens, from the state S before the chunk (rows i, j of the chunk, m tokens of it real):
//     P_ij = g^{i-j} (q_i . k_j) for j <= i, else 0
//     o_i  = scale (g^{i+1} S q_i + sum_j P_ij v_j)
//     S'   = g^m S + sum_j (g^{m-1-j} v_j) k_j^T
// Only powers g^e with e >= 0 are formed, so that no decay overflows.
//
// One CTA holds a tile of 64 value dimensions of one (prompt, head) and walks its chunks; all four products run on tcgen05:
//     scores  [128 i x 128 j]   Q K^T                  both K-major, as TMA brings them (128-byte swizzle)
//     inter   [128 i x 64 dv]   Q S^T                  S as bf16 hi + lo in shared memory, rows dk
//     update  [DK dk x 64 dv]   K^T V'                 K read M-major, V' = g^{m-1-j} v_j as 2 or 3 bf16 parts
//     intra   [128 i x 64 dv]   P V                    P bf16 in tensor memory (over the scores), V N-major as it came
// The state itself stays in fp32 registers (thread = dk, 64 dv) and never passes through fewer bits: an update adds the
// product to it, and what is rounded are operands.  hi + lo is 16 bits of S in o, which is bf16.  v g^e is rounded to
// 2^-17 of each term for a bf16 pool and, in three parts, to 2^-25 for an fp32 pool, whose states keep fp32's digits.  P is
// rounded to bf16 as o is: its rounding errors are those of single terms of a sum.
//
// Ten warps: 0-3 form P from the scores and write o (thread = row i), 4-7 form V' from V and the state (thread = token, then
// dk), 8 brings the tiles by TMA (two stages), 9 issues the products.  The order of products in a step, inter, update, intra and
// the next chunk's scores, leaves the state's conversion (the only serial chain between chunks) the time of the last two.
//
// Few prompts and heads leave SMs without work: then prompts are cut into pieces (linear_split), a first launch forms what
// each piece adds to the state (K and V only), and the second starts every piece from the sum of those before it.
#include <atomic>
#include <cstring>
#include <type_traits>

#include "gdn_tcgen05.cuh"

namespace gdn {

namespace {

constexpr int kLC = 128;   // tokens of a chunk
constexpr int kLDv = 64;   // value dimensions of a CTA
constexpr int kLThreads = 320;
constexpr uint32_t kLPolls = GDN_WAIT_POLLS;

enum { kFull = 0, kEmpty = 2, kScFull = 4, kIFull, kUFull, kOFull, kDrain, kPReady, kVReady, kLReady, kSReady, kOFree, kNumLBars };
// tensor memory: scores (P over them) of two chunks, intra, inter, update
constexpr uint32_t kScCol = 0, kO1Col = 256, kO2Col = 320, kUCol = 384, kLCols = 512;

template <int DK>
struct LinearPlan {
    static constexpr uint32_t BOX = kLC * 128;             // 64 columns of 128 rows
    static constexpr uint32_t QK = DK / 64 * BOX;
    static constexpr uint32_t Q_OFF = 0, K_OFF = QK, V_OFF = 2 * QK, STAGE = 2 * QK + BOX;
    static constexpr uint32_t VP_OFF = 2 * STAGE;          // V' hi, then its second part
    static constexpr uint32_t SH_OFF = VP_OFF + 2 * BOX;   // S hi, then lo: DK rows of 128 bytes each
    static constexpr uint32_t SPART = DK * 128;
    // the third part of V' lies over S (and behind it): the product that reads S is complete before it is written
    static constexpr uint32_t S_BYTES = 2 * SPART > BOX ? 2 * SPART : BOX;
    static constexpr uint32_t PW_OFF = SH_OFF + S_BYTES;   // g^0 .. g^128
    static constexpr uint32_t BAR_OFF = PW_OFF + 132 * 4;
    static constexpr uint32_t END = BAR_OFF + 8 * kNumLBars + 32;
    static constexpr uint32_t BYTES = END + 1024;          // the base is aligned to 1024
    static_assert(BYTES <= 232448, "fits one SM");
};

struct LinearMaps {
    CUtensorMap q, k, v;
};

// (x, y) as bf16 in one word, and what that leaves of them
__device__ __forceinline__ uint32_t take_bf16(float2& x) {
    const uint32_t w = bf16x2_bits(x.x, x.y);
    x = __ffma2_rn(bf16x2_to_float2(w), make_float2(-1.f, -1.f), x);  // exact
    return w;
}

// kState: the first launch of cut prompts (what a piece adds to the state; no queries, no outputs)
template <int DK, typename StT, bool kState>
__global__ void __launch_bounds__(kLThreads, 1)
    gdn_linear_prefill_kernel(const LinearParams p, const __grid_constant__ LinearMaps maps, const int piece, float* ws) {
    constexpr int NP = std::is_same<StT, float>::value ? 3 : 2;  // parts of V'
    using PL = LinearPlan<DK>;
    const int ndv = (p.DV + kLDv - 1) / kLDv;
    const int item = blockIdx.x, tile = item % ndv, h = item / ndv % p.HV, b = item / (ndv * p.HV);
    const int dv0 = tile * kLDv, hk = h / (p.HV / p.HK);
    const int tid = threadIdx.x, warp = tid >> 5, lt = tid & 127;

    const int slot = p.indices[b];
    const int out = p.out_indices != nullptr ? p.out_indices[b] : slot;
    const bool reporter = !kState && p.err != nullptr && tid == 0;
    if (slot == -1) return;
    if (slot < -1 || slot >= p.num_slots || out < -1 || out >= p.num_slots) {
        if (reporter) atomicOr(p.err, GDN_ERRBIT_INDEX);
        return;
    }
    const int lo = p.cu_seqlens[b], hi = p.cu_seqlens[b + 1];
    if (lo < 0 || hi < lo || hi > p.N) {
        if (reporter) atomicOr(p.err, GDN_ERRBIT_SEQLEN);
        return;
    }
    const int all = hi - lo;
    // this CTA's piece: tokens first .. first + n - 1 of the prompt
    const int64_t first64 = (int64_t)blockIdx.y * piece;
    if (first64 > 0 && first64 >= all) return;
    const int first = (int)first64;
    const int n = piece > 0 && all - first > piece ? piece : all - first;
    const bool last = first + n == all, cut = n < all;
    if (kState && last) return;  // nothing starts behind it
    if (all == 0 && (out < 0 || out == slot)) return;
    const bool init = p.has_init == nullptr || p.has_init[b] != 0;
    const int nch = (n + kLC - 1) / kLC;
    const int tok0 = lo + first;

    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), pad = ((raw + 1023u) & ~1023u) - raw;
    unsigned char* sm = smem_raw + pad;
    const uint32_t base = raw + pad;
    auto bar = [&](int i) -> uint32_t { return base + PL::BAR_OFF + 8u * (uint32_t)i; };
    float* pw = reinterpret_cast<float*>(sm + PL::PW_OFF);
    volatile int* fail = reinterpret_cast<volatile int*>(sm + PL::BAR_OFF + 8 * kNumLBars);
    volatile int* odd = fail + 1;  // [2]: c + 1 where V of chunk c (by its parity) holds an infinity or NaN
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + PL::BAR_OFF + 8 * kNumLBars + 16);
    const float ld = p.log_decay[h];

    if (warp == 0) tmem_alloc(smem_u32(tmem_slot), kLCols);
    if (tid == 32) {
        for (int i = 0; i < 2; ++i) mbar_init(bar(kFull + i), 1), mbar_init(bar(kEmpty + i), kState ? 1 : 1 + 128);
        for (int i = kScFull; i < kPReady; ++i) mbar_init(bar(i), 1);       // arrivals of products
        for (int i = kPReady; i < kNumLBars; ++i) mbar_init(bar(i), 128);  // of a group of threads
        fence_mbar_init();
        fail[0] = odd[0] = odd[1] = 0;
    }
    if (tid < kLC + 1) pw[tid] = tid == 0 ? 1.f : (float)exp((double)tid * (double)ld);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    auto stage = [&](int c) -> uint32_t { return (uint32_t)(c & 1) * PL::STAGE; };
    // bounded: a wait that runs out marks the CTA as failed, which ends every other wait of it
    auto wait = [&](int i, uint32_t parity) -> bool {
        for (uint32_t k = 0; k < kLPolls; ++k) {
            if (mbar_try_wait(bar(i), parity)) return true;
            if ((k & 255u) == 255u && *fail != 0) return false;
        }
        *fail = 1;
        return false;
    };
    auto warp_wait = [&](int i, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(i, parity)); };

    if (warp < 4 && !kState) {
        // ============ thread = row i of the chunk: P from the scores, o from the two products ============
        float r[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = pw[e];
        const float gi = pw[lt + 1];
        auto write_o = [&](int c) -> bool {
            if (!warp_wait(kOFull, (uint32_t)c & 1u)) return false;
            tc_fence_after();
            const int m = min(kLC, n - c * kLC);
            __nv_bfloat16* dst =
                static_cast<__nv_bfloat16*>(p.o) + ((int64_t)(tok0 + c * kLC + lt) * p.HV + h) * p.DV + dv0;
            const bool slow = odd[c & 1] == c + 1;
#pragma unroll 1
            for (int c0 = 0; c0 < kLDv; c0 += 32) {
                float a[32], x[32];
#pragma unroll
                for (int e = 0; e < 32; e += 16) {
                    tmem_ld16(lane_base + kO1Col + c0 + e, a + e);
                    tmem_ld16(lane_base + kO2Col + c0 + e, x + e);
                }
                tmem_wait_ld();
                if (slow) {
                    // 0 times an infinity of a later token must not reach this row: its own tokens alone, one by one
#pragma unroll
                    for (int e = 0; e < 32; ++e) a[e] = 0.f;
#pragma unroll 1
                    for (int j0 = 0; j0 < kLC; j0 += 32) {
                        float pp[16];  // 32 weights, two a word
                        tmem_ld16(lane_base + kScCol + (uint32_t)(c & 1) * 128 + j0 / 2, pp);
                        tmem_wait_ld();
#pragma unroll 1
                        for (int jj = 0; jj < 32; ++jj) {
                            float wj = 0.f;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (e == jj / 2) wj = (jj & 1) ? bf16x2_to_float2(__float_as_uint(pp[e])).y
                                                               : bf16x2_to_float2(__float_as_uint(pp[e])).x;
                            const int j = j0 + jj;
                            if (j > lt || j >= m) continue;
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                const uint4 q4 =
                                    *reinterpret_cast<const uint4*>(sm + stage(c) + PL::V_OFF + sw128(kLC, j, (c0 + e) / 8));
                                const uint32_t vw[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const float2 f = bf16x2_to_float2(vw[u]);
                                    a[e + 2 * u] = fmaf(wj, f.x, a[e + 2 * u]);
                                    a[e + 2 * u + 1] = fmaf(wj, f.y, a[e + 2 * u + 1]);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 y = __fmul2_rn(
                            make_float2(p.scale, p.scale),
                            __ffma2_rn(make_float2(gi, gi), make_float2(x[e + 2 * u], x[e + 2 * u + 1]),
                                       make_float2(a[e + 2 * u], a[e + 2 * u + 1])));
                        w[u] = bf16x2_bits(y.x, y.y);
                    }
                    if (lt < m && dv0 + c0 + e < p.DV)
                        *reinterpret_cast<uint4*>(dst + c0 + e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            tc_fence_before();
            mbar_arrive(bar(kOFree));
            mbar_arrive(bar(kEmpty + (c & 1)));
            return true;
        };
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            if (c > 0 && !write_o(c - 1)) {
                ok = false;
                break;
            }
            if (!warp_wait(kScFull, (uint32_t)c & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sc = lane_base + kScCol + (uint32_t)(c & 1) * 128;
#pragma unroll 1
            for (int jb = 0; jb < 8; ++jb) {  // 16 columns at a time; P lies over scores that have been read
                uint32_t w[8];
                if (jb < 2 * warp + 2) {
                    float s[16];
                    tmem_ld16(sc + 16 * jb, s);
                    tmem_wait_ld();
                    if (jb < 2 * warp) {  // below the diagonal for every row of the warp
                        const float f = pw[lt - (16 * jb + 15)];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 g2 = __fmul2_rn(make_float2(f, f), make_float2(r[15 - 2 * e], r[14 - 2 * e]));
                            const float2 y = __fmul2_rn(g2, make_float2(s[2 * e], s[2 * e + 1]));
                            w[e] = bf16x2_bits(y.x, y.y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int d = lt - (16 * jb + 2 * e);  // i - j of the first of the two
                            const float y0 = d >= 0 ? s[2 * e] * pw[max(d, 0)] : 0.f;
                            const float y1 = d >= 1 ? s[2 * e + 1] * pw[max(d - 1, 0)] : 0.f;
                            w[e] = bf16x2_bits(y0, y1);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                }
                tmem_st8(sc + 8 * jb, w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(kPReady));
        }
        if (ok && nch > 0) write_o(nch - 1);
    } else if (warp >= 4 && warp < 8) {
        // ============ thread = token of the chunk (V'), then dk (the state) ============
        const bool mine = lt < DK;
        const int64_t row = ((int64_t)h * p.DV + dv0) * DK + lt;  // of [HV, DV, DK]: dv0's row, column dk
        const int64_t slot_elems = (int64_t)p.HV * p.DV * DK;
        float2 S[kLDv / 2];
#pragma unroll
        for (int e = 0; e < kLDv / 2; ++e) S[e] = make_float2(0.f, 0.f);
        float* wsp = ws != nullptr ? ws + (int64_t)item * gridDim.y * (kLDv * DK) + lt : nullptr;
        // pieces after the first start from the states that the first launch left; it also kept the initial state of a cut
        // prompt, whose slot the prompt's last piece may have overwritten
        const bool from_ws = !kState && cut;
        if (mine) {
            if (from_ws) {
                const int np = blockIdx.y == 0 ? 0 : 1;
                const float gp = (float)exp((double)piece * (double)ld);
                for (int s = np; s <= (int)blockIdx.y; ++s) {
                    const float* src = wsp + (int64_t)s * (kLDv * DK);
                    const float f = s == np ? 0.f : gp;
#pragma unroll
                    for (int e = 0; e < kLDv / 2; ++e) {
                        const float2 u = make_float2(src[(2 * e) * DK], src[(2 * e + 1) * DK]);
                        S[e] = s == np ? u : __ffma2_rn(make_float2(f, f), S[e], u);
                    }
                }
            } else if (init && blockIdx.y == 0) {
                const StT* src = static_cast<const StT*>(p.pool) + (int64_t)slot * slot_elems + row;
#pragma unroll
                for (int e = 0; e < kLDv; ++e) {
                    const float x = dv0 + e < p.DV ? to_f32(src[(int64_t)e * DK]) : 0.f;
                    if (e & 1) S[e / 2].y = x; else S[e / 2].x = x;
                }
            }
            if (kState && blockIdx.y == 0) {
#pragma unroll
                for (int e = 0; e < kLDv; ++e) wsp[e * DK] = (e & 1) ? S[e / 2].y : S[e / 2].x;
            }
        }
        auto put_state = [&]() {  // S as hi and lo, rows dk
            if (mine) {
#pragma unroll
                for (int c8 = 0; c8 < 8; ++c8) {
                    uint32_t hw[4], lw[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float2 x = S[4 * c8 + u];
                        hw[u] = take_bf16(x);
                        lw[u] = bf16x2_bits(x.x, x.y);
                    }
                    const uint32_t at = sw128(DK, lt, c8);
                    *reinterpret_cast<uint4*>(sm + PL::SH_OFF + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                    *reinterpret_cast<uint4*>(sm + PL::SH_OFF + PL::SPART + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(kSReady));
        };
        bool ok = true;
        if (!kState && nch > 0) put_state();
        for (int c = 0; c < nch; ++c) {
            ok = warp_wait(kFull + (c & 1), (uint32_t)(c >> 1) & 1u);
            if (!ok) break;
            const int m = min(kLC, n - c * kLC);
            unsigned char* vt = sm + stage(c) + PL::V_OFF;
            const bool real = lt < m;
            const float f = real ? pw[m - 1 - lt] : 0.f;
            float2 third[NP == 3 ? kLDv / 2 : 1];
            float2 probe = make_float2(0.f, 0.f);
            if (!real) {  // rows behind the prompt's last token belong to others, or to nobody
#pragma unroll
                for (int c8 = 0; c8 < DK / 8; ++c8)
                    *reinterpret_cast<uint4*>(sm + stage(c) + PL::K_OFF + sw128(kLC, lt, c8)) = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8) {
                const uint32_t at = sw128(kLC, lt, c8);
                uint4 v4 = make_uint4(0, 0, 0, 0);
                if (real)
                    v4 = *reinterpret_cast<const uint4*>(vt + at);
                else
                    *reinterpret_cast<uint4*>(vt + at) = v4;
                const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float2 v2 = bf16x2_to_float2(vw[u]);
                    probe = __ffma2_rn(v2, make_float2(0.f, 0.f), probe);  // 0 unless one is not finite
                    float2 x = __fmul2_rn(make_float2(f, f), v2);
                    hw[u] = take_bf16(x);
                    lw[u] = bf16x2_bits(x.x, x.y);
                    if constexpr (NP == 3) {
                        (void)take_bf16(x);
                        third[4 * c8 + u] = x;
                    }
                }
                *reinterpret_cast<uint4*>(sm + PL::VP_OFF + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                *reinterpret_cast<uint4*>(sm + PL::VP_OFF + PL::BOX + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
            }
            if (!(probe.x == 0.f && probe.y == 0.f)) odd[c & 1] = c + 1;
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(kVReady));
            if constexpr (NP == 3) {
                if (!kState) {
                    ok = warp_wait(kIFull, (uint32_t)c & 1u);
                    if (!ok) break;
                }
#pragma unroll
                for (int c8 = 0; c8 < 8; ++c8) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) w[u] = bf16x2_bits(third[4 * c8 + u].x, third[4 * c8 + u].y);
                    *reinterpret_cast<uint4*>(sm + PL::SH_OFF + sw128(kLC, lt, c8)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(kLReady));
            }
            ok = warp_wait(kUFull, (uint32_t)c & 1u);
            if (!ok) break;
            tc_fence_after();
            const float gm = pw[m];
#pragma unroll
            for (int c0 = 0; c0 < kLDv; c0 += 16) {
                float u[16];
                tmem_ld16(lane_base + kUCol + c0, u);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    S[c0 / 2 + e] = __ffma2_rn(make_float2(gm, gm), S[c0 / 2 + e], make_float2(u[2 * e], u[2 * e + 1]));
            }
            tc_fence_before();
            if (!kState && c + 1 < nch) put_state();
        }
        if (ok && mine) {
            if constexpr (kState) {
                float* dst = wsp + (int64_t)(blockIdx.y + 1) * (kLDv * DK);
#pragma unroll
                for (int e = 0; e < kLDv; ++e) dst[e * DK] = (e & 1) ? S[e / 2].y : S[e / 2].x;
            } else if (last && out >= 0) {
                StT* dst = static_cast<StT*>(p.pool) + (int64_t)out * slot_elems + row;
#pragma unroll
                for (int e = 0; e < kLDv; ++e) {
                    const float x = (e & 1) ? S[e / 2].y : S[e / 2].x;
                    if (dv0 + e < p.DV) {
                        if constexpr (std::is_same<StT, float>::value)
                            dst[(int64_t)e * DK] = x;
                        else
                            dst[(int64_t)e * DK] = __float2bfloat16_rn(x);
                    }
                }
            }
        }
    } else if (tid == 256) {
        // ============ tiles by TMA ============
        constexpr uint32_t bytes = (kState ? PL::QK : 2 * PL::QK) + PL::BOX;
        int issued = 0;
        for (int c = 0; c < nch; ++c) {
            if (c >= 2 && !wait(kEmpty + (c & 1), (uint32_t)((c - 2) >> 1) & 1u)) break;
#ifdef GDN_TEST_MISSING_COPY
            // test build: the first chunk of the first item is never loaded nor arrived on: its wait runs out
            if (item == 0 && blockIdx.y == 0 && c == 0) break;
#endif
            const uint32_t full = bar(kFull + (c & 1)), st = base + stage(c);
            mbar_arrive_expect_tx(full, bytes);
#pragma unroll
            for (int j = 0; j < DK / 64; ++j) {
                tma_load_3d(st + PL::K_OFF + j * PL::BOX, &maps.k, 64 * j, hk, tok0 + c * kLC, full);
                if (!kState) tma_load_3d(st + PL::Q_OFF + j * PL::BOX, &maps.q, 64 * j, hk, tok0 + c * kLC, full);
            }
            tma_load_3d(st + PL::V_OFF, &maps.v, dv0, h, tok0 + c * kLC, full);
            issued = c + 1;
        }
        for (int c = max(0, issued - 2); c < issued; ++c)  // copies in flight land before the CTA leaves
            mbar_wait_bounded(bar(kFull + (c & 1)), (uint32_t)(c >> 1) & 1u, kLPolls);
    } else if (tid == 288) {
        // ============ products ============
        bool any = false;
        auto scores = [&](int c) -> bool {
            if (!wait(kFull + (c & 1), (uint32_t)(c >> 1) & 1u)) return false;
            // the rows behind the last token are cleared first
            if (n - c * kLC < kLC && !wait(kVReady, (uint32_t)c & 1u)) return false;
            tc_fence_after();
            const uint32_t st = base + stage(c);
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                const uint32_t off = (uint32_t)(ks >> 2) * PL::BOX + (uint32_t)(ks & 3) * 32u;
                umma_bf16(tmem + kScCol + (uint32_t)(c & 1) * 128, umma_desc_sw128(st + PL::Q_OFF + off),
                          umma_desc_sw128(st + PL::K_OFF + off), umma_idesc_bf16(kLC, kLC), ks > 0 ? 1u : 0u);
            }
            umma_commit(bar(kScFull));
            any = true;
            return true;
        };
        constexpr uint32_t kBn = 1u << 16, kAm = 1u << 15;  // B N-major, A M-major
        constexpr uint32_t id64 = umma_idesc_bf16(128, kLDv);
        bool ok = true;
        if (!kState && nch > 0) ok = scores(0);
        for (int c = 0; c < nch && ok; ++c) {
            const uint32_t st = base + stage(c);
            if constexpr (!kState) {
                ok = wait(kSReady, (uint32_t)c & 1u) && (c == 0 || wait(kOFree, (uint32_t)(c - 1) & 1u));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < DK / 16; ++ks) {
                        const uint32_t off = (uint32_t)(ks >> 2) * PL::BOX + (uint32_t)(ks & 3) * 32u;
                        umma_bf16(tmem + kO2Col, umma_desc_sw128(st + PL::Q_OFF + off),
                                  umma_desc_sw128_mn(base + PL::SH_OFF + part * PL::SPART + ks * 2048u, PL::BOX), id64 | kBn,
                                  part + ks > 0 ? 1u : 0u);
                    }
                umma_commit(bar(kIFull));
            }
            if (!wait(kVReady, (uint32_t)c & 1u) || (kState && !wait(kFull + (c & 1), (uint32_t)(c >> 1) & 1u))) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < NP; ++part) {
                if (part == 2) {
                    ok = wait(kLReady, (uint32_t)c & 1u);
                    if (!ok) break;
                }
                const uint32_t vp = base + (part < 2 ? PL::VP_OFF + part * PL::BOX : PL::SH_OFF);
#pragma unroll
                for (int ks = 0; ks < kLC / 16; ++ks)
                    umma_bf16(tmem + kUCol, umma_desc_sw128_mn(st + PL::K_OFF + ks * 2048u, PL::BOX),
                              umma_desc_sw128_mn(vp + ks * 2048u, PL::BOX), id64 | kBn | kAm, part + ks > 0 ? 1u : 0u);
            }
            any = true;
            if (!ok) break;
            umma_commit(bar(kUFull));
            if constexpr (kState) {
                umma_commit(bar(kEmpty + (c & 1)));
            } else {
                ok = wait(kPReady, (uint32_t)c & 1u);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kLC / 16; ++ks)
                    umma_bf16_ta(tmem + kO1Col, tmem + kScCol + (uint32_t)(c & 1) * 128 + 8 * ks,
                                 umma_desc_sw128_mn(st + PL::V_OFF + ks * 2048u, PL::BOX), id64 | kBn, ks > 0 ? 1u : 0u);
                umma_commit(bar(kOFull));
                umma_commit(bar(kEmpty + (c & 1)));
                if (c + 1 < nch) ok = scores(c + 1);
            }
        }
        if (any) {  // every product is complete before the tensor memory is released
            umma_commit(bar(kDrain));
            mbar_wait_bounded(bar(kDrain), 0u, kLPolls);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *fail != 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, kLCols);
}

int linear_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 152;
    }
    return sms;
}

// Tokens of a piece (a multiple of the chunk), 0 where prompts stay whole.  Cutting reads K and V once more, so it must at
// least double the SMs at work.
int linear_split(int B, int N, int HV, int DV) {
    const int64_t items = (int64_t)B * HV * ((DV + kLDv - 1) / kLDv);
    if (items == 0 || N == 0) return 0;
    const int64_t times = linear_sms() / items;  // pieces that fill the GPU once
    if (times < 2) return 0;
    const int64_t chunks = ((int64_t)N / B + kLC - 1) / kLC;
    const int64_t per = (chunks + times - 1) / times > 4 ? (chunks + times - 1) / times : 4;
    if (2 * per > chunks) return 0;
    return (int)(per * kLC);
}

bool encode_rows(CUtensorMap* map, const void* ptr, int cols, int heads, int n) {
    const EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)heads * cols * 2};
    const cuuint32_t box[3] = {64, 1, kLC};
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, typename StT, bool kState>
cudaError_t launch_one(const LinearParams& p, const LinearMaps& m, int piece, int pieces, float* ws, cudaStream_t s) {
    using PL = LinearPlan<DK>;
    auto kernel = gdn_linear_prefill_kernel<DK, StT, kState>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // the attribute is per device: set once for each
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PL::BYTES);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_acq_rel);
    }
    const int64_t items = (int64_t)p.B * p.HV * ((p.DV + kLDv - 1) / kLDv);
    kernel<<<dim3((unsigned)items, (unsigned)pieces), kLThreads, PL::BYTES, s>>>(p, m, piece, ws);
    return cudaGetLastError();
}

template <int DK, typename StT>
cudaError_t launch_dk(const LinearParams& p, const LinearMaps& m, float* ws, cudaStream_t s) {
    const int piece = linear_split(p.B, p.N, p.HV, p.DV);
    const int pieces = piece > 0 ? (p.N + piece - 1) / piece : 1;
    if (pieces > 1) {
        const cudaError_t e = launch_one<DK, StT, true>(p, m, piece, pieces, ws, s);
        if (e != cudaSuccess) return e;
    }
    return launch_one<DK, StT, false>(p, m, piece, pieces, ws, s);
}

}  // namespace

int64_t linear_prefill_workspace(int B, int N, int HV, int DK, int DV) {
    if (DK != 64 && DK != 128) return 0;
    const int piece = linear_split(B, N, HV, DV);
    if (piece == 0) return 0;
    return (int64_t)((N + piece - 1) / piece) * B * HV * ((DV + kLDv - 1) / kLDv) * kLDv * DK * 4;
}

bool launch_linear_prefill(const LinearParams& p, bool qkv_bf16, bool state_bf16, float* ws, cudaStream_t s, cudaError_t& err) {
    const int64_t items = (int64_t)p.B * p.HV * ((p.DV + kLDv - 1) / kLDv);
    if ((p.DK != 64 && p.DK != 128) || !qkv_bf16 || !p.out_bf16 || !p.v_vec || (reinterpret_cast<uintptr_t>(p.o) & 15u) != 0 ||
        p.N == 0 || items > 0x7fffffff)
        return false;
    LinearMaps m;
    std::memset(&m, 0, sizeof m);
    if (!encode_rows(&m.q, p.q, p.DK, p.HK, p.N) || !encode_rows(&m.k, p.k, p.DK, p.HK, p.N) ||
        !encode_rows(&m.v, p.v, p.DV, p.HV, p.N))
        return false;
    if (p.DK == 64)
        err = state_bf16 ? launch_dk<64, __nv_bfloat16>(p, m, ws, s) : launch_dk<64, float>(p, m, ws, s);
    else
        err = state_bf16 ? launch_dk<128, __nv_bfloat16>(p, m, ws, s) : launch_dk<128, float>(p, m, ws, s);
    return true;
}

}  // namespace gdn
