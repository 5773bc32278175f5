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
//     inter   [128 i x 64 dv]   Q S^T                  S as bf16 in shared memory, rows dk
//     update  [DK dk x 64 dv]   K^T V'                 K read M-major, V' = g^{m-1-j} v_j as 2 or 3 bf16 parts
//     intra   [128 i x 64 dv]   P V                    P bf16 in tensor memory (over the scores), V N-major as it came
// The state itself stays in fp32 registers (thread = dk, 32 dv) and never passes through fewer bits: an update adds the product
// to it, and what is rounded are operands.  S is rounded to bf16 on its way into o, as o is, and so is P: the errors are those of
// single terms of a sum.  v g^e, which the pool keeps, is good to 2^-16 of each term in two bf16 parts for a bf16 pool and to 2^-24
// in three for an fp32 pool, whose states keep fp32's digits.
//
// Three groups of eight warps: the first forms P from the scores (thread = row i and a half of the columns), the second keeps the
// state (thread = dk and 32 dv), the third forms V' from V (thread = token and 32 dv) and takes o from the products (thread = row
// i and 32 dv).  Warp 24 brings the tiles by TMA (two stages), 25 issues the products, 26 stores o by TMA, 27 says when V has been
// read.  A group's work on a chunk is a few hundred dependent instructions, at which one warp issues every sixth cycle or so: eight
// warps a group take half the time of four.  For the same reason code is kept short (unrolled to 95 KB, the warps waited for
// instructions).  The only serial chains between chunks are state -> inter -> state and V' -> update -> state; the scores of the
// next chunk and the intra product fill the tensor cores meanwhile.
//
// P and S as bf16 take o to 0.0023 of itself from 64-bit arithmetic, where its own rounding alone leaves 0.0017.  P in two parts, which its
// place in tensor memory has room for, is 8 more products a chunk: 0.0020, for 419 us instead of 392 in the first case below and 141 instead of 133
// in the second; S in two parts does not fit beside three of V'.
//
// Waits of a warp go by votes (warp_wait): after a lane-by-lane wait the warp can stay in parts, and each would issue its products and commits.
// Where V or k of a chunk holds what is not finite, o sums P V and the state its tokens one by one: about 66 us a chunk.
//
// Measured (D 128, HK 16, HV 32, bf16 pool): 7 prompts of 8192 and an empty one 394 us (3.6 TB/s, 305 TFLOP/s of the recurrence's 4 DK DV a token;
// three waves of CTAs), 8 of 8192 511 (four), 4 of 2048 76; a step of one chunk and 64 dv takes about 3700 cycles, of which the products run
// 2000 and their issue takes 2770, and a CTA's start and end 9 us.  Two warps issuing two products each measured the same.
//
// Few prompts and heads leave SMs without work: then prompts are cut into pieces (linear_split), a first launch forms what
// each piece adds to the state (K and V only), and the second starts every piece from the sum of those before it (one prompt of
// 16384, fp32 pool, HV 16: 133 us on 128 CTAs; whole, with 76 heads on 152 CTAs, 337).
#include <atomic>
#include <cfloat>
#include <cstring>
#include <type_traits>

#include "gdn_tcgen05.cuh"

namespace gdn {

namespace {

constexpr int kLC = 128;   // tokens of a chunk
constexpr int kLDv = 64;   // value dimensions of a CTA
constexpr int kLGroup = 256;                 // threads of a group
constexpr int kLThreads = 3 * kLGroup + 128;
constexpr int kLHalf = kLDv / 2;              // value dimensions of a thread
constexpr uint32_t kLPolls = GDN_WAIT_POLLS;

// barriers (the first ones: one for each of two stages or score buffers); a stage's K and Q are free before its V
enum { kQkFull = 0, kVFull = 2, kEmptyQk = 4, kEmptyV = 6, kScFull = 8, kIFull = 10, kUFull, kOFull = kUFull + 2, kStFree, kDrain, kPReady, kVReady = kPReady + 2, kStaged = kVReady + 2, kUFree = kStaged + 2,
       kSReady = kUFree + 2, kOFree, kNumLBars };
// tensor memory: scores (P over them) of two chunks, intra, inter, update
constexpr uint32_t kScCol = 0, kO1Col = 256, kO2Col = 320, kUCol = 384, kLCols = 512;

template <int DK, int NP>
struct LinearPlan {
    static constexpr uint32_t BOX = kLC * 128;             // 64 columns of 128 rows
    static constexpr uint32_t QK = DK / 64 * BOX;
    static constexpr uint32_t Q_OFF = 0, K_OFF = QK, V_OFF = 2 * QK, STAGE = 2 * QK + BOX;
    static constexpr uint32_t VP_OFF = 2 * STAGE;          // the parts of V'
    static constexpr uint32_t SH_OFF = VP_OFF + NP * BOX;  // S: DK rows of 128 bytes
    // o on its way out: a place of its own where there is room (all but fp32 pools of DK = 128), else where V was
    static constexpr bool OWN = DK == 64 || NP == 2;
    static constexpr uint32_t O_OFF = SH_OFF + DK * 128;
    static constexpr uint32_t PW_OFF = O_OFF + (OWN ? BOX : 0) + 128;  // g^0 .. g^128, behind 32 floats that are read and not used
    static constexpr uint32_t BAR_OFF = PW_OFF + 132 * 4;
    static constexpr uint32_t END = BAR_OFF + 8 * kNumLBars + 48;
    static constexpr uint32_t BYTES = END + 1024;          // the base is aligned to 1024
    static_assert(BYTES <= 232448, "fits one SM");
    // The first launch of cut prompts has no queries and no o: the parts of V' of odd chunks lie there, so that one chunk's V' is formed
    // beside the last one's update.
    static constexpr __host__ __device__ uint32_t vp(bool odd, int e) {
        return !odd ? VP_OFF + e * BOX : DK == 128 ? (e < 2 ? Q_OFF + e * BOX : STAGE + Q_OFF) : e < 2 ? Q_OFF + e * STAGE : O_OFF;
    }
};

struct LinearMaps {
    CUtensorMap q, k, v, o;
};

// (x, y) as bf16 in one word, and what that leaves of them
__device__ __forceinline__ uint32_t take_bf16(float2& x) {
    const uint32_t w = bf16x2_bits(x.x, x.y);
    x = __ffma2_rn(bf16x2_to_float2(w), make_float2(-1.f, -1.f), x);  // exact
    return w;
}

// One lane of the warp, chosen by the hardware
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {  // without waiting
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// What a wait of one thread does after its first try, out of line: the code that runs once a chunk stays short
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, uint32_t fail) {
    for (uint32_t k = 0; k < kLPolls; ++k) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((k & 255u) == 255u) {
            int f;
            asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(f) : "r"(fail) : "memory");
            if (f != 0) return false;
        }
    }
    asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(fail) : "memory");
    return false;
}
// The same of a whole warp, each lane for its barrier.  Every branch goes by a vote: products, commits and tensor memory's loads and stores
// are instructions of the warp, and a warp whose lanes left a wait one after the other would issue them once for each part of it.
__device__ __noinline__ bool warp_wait_more(uint32_t bar, uint32_t parity, uint32_t fail) {
    for (uint32_t k = 0; k < kLPolls; ++k) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((k & 255u) == 255u) {
            int f;
            asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(f) : "r"(fail) : "memory");
            if (__any_sync(0xffffffffu, f != 0)) return false;
        }
    }
    asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(fail) : "memory");
    return false;
}

// Where a CTA's tokens are, in shared memory for add_tokens
struct Place {
    int tok0, h, hk, dv0;
};
// What the m tokens of chunk c give to a thread's 32 columns of the state, which lie in tensor memory: column e += sum_j g^(m-1-j) v_j[e] k_j,
// token by token in fp32.  For chunks that hold what is not finite; out of line, since the state's threads have no registers for it.
template <int DK>
__device__ __noinline__ void add_tokens(const LinearParams& p, const volatile Place* at, const float* pw, uint32_t columns, int c, int m) {
    const int64_t tok = at->tok0 + c * kLC;
    const int first = at->dv0 + kLHalf * ((threadIdx.x >> 7) & 1), dv = p.DV - first, kstep = p.HK * DK;
    const int64_t vstep = (int64_t)p.HV * p.DV;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + (tok * p.HK + at->hk) * DK + (threadIdx.x & 127);
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + (tok * p.HV + at->h) * p.DV + first;
#pragma unroll 1
    for (int c0 = 0; c0 < kLHalf; c0 += 16) {
        float x[16];
        tmem_ld16(columns + c0, x);
        tmem_wait_ld();
#pragma unroll 1
        for (int j = 0; j < m; ++j) {
            const float k1 = __bfloat162float(k[(int64_t)j * kstep]), f = pw[m - 1 - j];
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                if (c0 + e >= dv) break;  // DV is a multiple of 8
                const uint4 v4 = *reinterpret_cast<const uint4*>(v + j * vstep + c0 + e);
                const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {  // v k first: where it is not finite it stays so, whatever f is
                    const float2 v2 = bf16x2_to_float2(vw[u]);
                    x[e + 2 * u] = fmaf(f, v2.x * k1, x[e + 2 * u]);
                    x[e + 2 * u + 1] = fmaf(f, v2.y * k1, x[e + 2 * u + 1]);
                }
            }
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(x[e]);
        tmem_st8(columns + c0, w);
        tmem_st8(columns + c0 + 8, w + 8);
    }
    tmem_wait_st();
}

// kState: the first launch of cut prompts (what a piece adds to the state; no queries, no outputs)
template <int DK, typename StT, bool kState>
__global__ void __launch_bounds__(kLThreads, 1)
    gdn_linear_prefill_kernel(const __grid_constant__ LinearParams p, const __grid_constant__ LinearMaps maps, const int piece, float* ws) {
    constexpr int NP = std::is_same<StT, float>::value ? 3 : 2;  // parts of V'
    using PL = LinearPlan<DK, NP>;
    const int ndv = (p.DV + kLDv - 1) / kLDv;
    const int item = blockIdx.x, tile = item % ndv, h = item / ndv % p.HV, turn = item / (ndv * p.HV);
    const int dv0 = tile * kLDv, hk = h / (p.HV / p.HK);
    const int tid = threadIdx.x, warp = __reduce_min_sync(0xffffffffu, tid >> 5), lt = tid & 127;
    const int hf = (warp >> 2) & 1, wl = warp & 3;  // half of a group, and the warp's quarter of the lanes

    // Everything that tells what to do is asked for at once.  Of up to 32 whole prompts a lane asks for one each, and the longest is
    // taken first, so that no long one is left for the end.  (HV 32, D 64, fp32 pool, in graph replays, against the order of the lanes: two draws
    // of 32 prompts of 17 to 2048 tokens 159 and 167 us against 168 and 178, of 8 of 17 to 8192 133 and 161 against 144 and 196; 32 of 1024 149 in
    // either.  33 prompts go in the lanes' order: a lane each is what a warp has.)
    const bool sorted = piece == 0 && p.B > 1 && p.B <= 32;
    int b = sorted ? min(tid & 31, p.B - 1) : turn;
    int slot = p.indices[b];
    int out = p.out_indices != nullptr ? p.out_indices[b] : slot;
    int lo = p.cu_seqlens[b], hi = p.cu_seqlens[b + 1];
    int has = p.has_init == nullptr ? 1 : p.has_init[b];
    if (sorted) {
        const uint32_t key = ((uint32_t)min(max(hi - lo, 0), (1 << 26) - 1) << 5) | (31u - (tid & 31));
        b = turn;
        if (!__all_sync(0xffffffffu, (key >> 5) == __shfl_sync(0xffffffffu, key >> 5, 0))) {
            int before = 0;
            for (int i = 0; i < p.B; ++i) before += __shfl_sync(0xffffffffu, key, i) > key;
            b = __ffs(__ballot_sync(0xffffffffu, (tid & 31) < p.B && before == turn)) - 1;
        }
    }
    const auto of_b = [&](int x) {  // the value of lane b where lanes have their own (a uniform register in either case)
        return __reduce_max_sync(0xffffffffu, !sorted || (tid & 31) == b ? x : INT32_MIN);
    };
    slot = of_b(slot), out = of_b(out), lo = of_b(lo), hi = of_b(hi), has = of_b(has);
    const bool init = has != 0;
    const float ld = p.log_decay[h];
    const bool reporter = !kState && p.err != nullptr && tid == 0;
    if (slot == -1) return;
    if (slot < -1 || slot >= p.num_slots || out < -1 || out >= p.num_slots) {
        if (reporter) atomicOr(p.err, GDN_ERRBIT_INDEX);
        return;
    }
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
    const int nch = n / kLC + (n % kLC != 0);
    const int tok0 = lo + first;

    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), pad = ((raw + 1023u) & ~1023u) - raw;
    unsigned char* sm = smem_raw + pad;
    const uint32_t base = raw + pad;
    auto bar = [&](int i) -> uint32_t { return base + PL::BAR_OFF + 8u * (uint32_t)i; };
    float* pw = reinterpret_cast<float*>(sm + PL::PW_OFF);
    volatile int* fail = reinterpret_cast<volatile int*>(sm + PL::BAR_OFF + 8 * kNumLBars);
    // [4]: c + 1 where V of chunk c (c mod 4) holds an infinity or NaN.  V' of chunk c + 4 is formed after o of chunk c + 2, which waits for the
    // storing warp to be past c + 1, and V of c + 4 is asked for when the releasing warp is past c + 2: a mark is read before it is written
    // over.  (With two, the storing warp could read that of c + 2 for c's.)
    volatile int* odd = fail + 1;
    volatile Place* const place = reinterpret_cast<volatile Place*>(sm + PL::BAR_OFF + 8 * kNumLBars + 32);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + PL::BAR_OFF + 8 * kNumLBars + 24);

    auto stage = [&](int c) -> uint32_t { return (uint32_t)(c & 1) * PL::STAGE; };
    auto load_qk = [&](int c) {
        const uint32_t st = base + stage(c), full = bar(kQkFull + (c & 1));
        mbar_arrive_expect_tx(full, kState ? PL::QK : 2 * PL::QK);
#pragma unroll
        for (int j = 0; j < DK / 64; ++j) {
            tma_load_3d(st + PL::K_OFF + j * PL::BOX, &maps.k, 64 * j, hk, tok0 + c * kLC, full);
            if (!kState) tma_load_3d(st + PL::Q_OFF + j * PL::BOX, &maps.q, 64 * j, hk, tok0 + c * kLC, full);
        }
    };
    auto load_v = [&](int c) {
        mbar_arrive_expect_tx(bar(kVFull + (c & 1)), PL::BOX);
        tma_load_3d(base + stage(c) + PL::V_OFF, &maps.v, dv0, h, tok0 + c * kLC, bar(kVFull + (c & 1)));
    };
    if (warp == 0) tmem_alloc(smem_u32(tmem_slot), kLCols);
    if (tid == 3 * kLGroup) {
        for (int i = kQkFull; i < kPReady; ++i)  // of copies and products; V is read by the intra product and by V' (kState: by V' alone)
            mbar_init(bar(i), (i & ~1) != kEmptyV ? 1 : kState ? kLGroup : PL::OWN ? 2 : 1);
        for (int i = kPReady; i < kNumLBars; ++i) mbar_init(bar(i), kLGroup);                                         // of a group of threads
        fence_mbar_init();
        fence_proxy_async_smem();
        fail[0] = odd[0] = odd[1] = odd[2] = odd[3] = 0;
        place->tok0 = tok0, place->h = h, place->hk = hk, place->dv0 = dv0;
#ifdef GDN_TEST_MISSING_COPY
        // test build: the first chunks of the first item are never loaded nor arrived on: their waits run out
        if (item > 0 || blockIdx.y > 0)
#endif
            for (int c = 0; c < min(nch, 2); ++c) load_qk(c), load_v(c);  // before anything else is set up
    }
    if (tid < 32) pw[tid - 32] = 0.f;
    if (tid < kLC + 1) pw[tid] = decay_power(ld, tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    auto u_col = [&](int c) -> uint32_t { return kState && (c & 1) ? kScCol : kUCol; };
    // bounded: a wait that runs out marks the CTA as failed, which ends every other wait of it
    auto wait = [&](int i, uint32_t parity) -> bool {  // of one thread
        return mbar_try_wait(bar(i), parity) || wait_more(bar(i), parity, smem_u32(const_cast<int*>(fail)));
    };
    auto warp_wait = [&](int i, uint32_t parity) -> bool {  // of a whole warp
        return __all_sync(0xffffffffu, mbar_try_wait(bar(i), parity)) ||
               warp_wait_more(bar(i), parity, smem_u32(const_cast<int*>(fail)));
    };

    if (warp < 8) {
        // ============ thread = row i of the chunk: P from the scores ============
        float r[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = pw[e];
        for (int c = 0; c < (kState ? 0 : nch); ++c) {
            if (!warp_wait(kScFull + (c & 1), (uint32_t)(c >> 1) & 1u)) break;
            tc_fence_after();
            const uint32_t sc = lane_base + kScCol + (uint32_t)(c & 1) * 128;
            // 16 columns at a time of this half's 64; P lies over this half's scores that have been read
#pragma unroll 1
            for (int jb = 4 * hf; jb < 4 * hf + 4; ++jb) {
                uint32_t w[8];
                float x[16];
                if (jb < 2 * wl + 2) {
                    tmem_ld16(sc + 16 * jb, x);
                    tmem_wait_ld();
                }
                if (jb < 2 * wl) {  // below the diagonal for every row of the warp
                    const float f = pw[lt - (16 * jb + 15)];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 g2 = __fmul2_rn(make_float2(f, f), make_float2(r[15 - 2 * e], r[14 - 2 * e]));
                        const float2 y = __fmul2_rn(g2, make_float2(x[2 * e], x[2 * e + 1]));
                        w[e] = bf16x2_bits(y.x, y.y);
                    }
                } else if (jb < 2 * wl + 2) {
                    const float* fp = pw + (lt - 16 * jb);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = lt - 16 * jb - 2 * e;  // i - j of the first of the two
                        // the factors are read in any case (32 floats in front of g^0 are there to be): no branch, a select
                        const float y0 = x[2 * e] * fp[-2 * e], y1 = x[2 * e + 1] * fp[-2 * e - 1];
                        w[e] = bf16x2_bits(d >= 0 ? y0 : 0.f, d >= 1 ? y1 : 0.f);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                }
                tmem_st8(sc + 64 * hf + 8 * (jb & 3), w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(kPReady + (c & 1)));
        }
    } else if (warp < 16) {
        // ============ thread = dk, half of the tile: the state ============
        const bool mine = 32 * wl < DK;  // of a warp
        const int dvh = dv0 + kLHalf * hf;                        // the thread's first value dimension
        const int64_t row = ((int64_t)h * p.DV + dvh) * DK + lt;  // of [HV, DV, DK]: its row, column dk
        const int64_t slot_elems = (int64_t)p.HV * p.DV * DK;
        float2 S[kLHalf / 2];
#pragma unroll
        for (int e = 0; e < kLHalf / 2; ++e) S[e] = make_float2(0.f, 0.f);
        float* wsp = ws != nullptr ? ws + (int64_t)item * gridDim.y * (kLDv * DK) + kLHalf * hf * DK + lt : nullptr;
        // pieces after the first start from the states that the first launch left; it also kept the initial state of a cut
        // prompt, whose slot the prompt's last piece may have overwritten
        const bool from_ws = !kState && cut;
        if (mine) {
            if (from_ws) {
                const int np = blockIdx.y == 0 ? 0 : 1;
                const float gp = decay_power(ld, piece);
                for (int s = np; s <= (int)blockIdx.y; ++s) {
                    const float* src = wsp + (int64_t)s * (kLDv * DK);
#pragma unroll
                    for (int e = 0; e < kLHalf / 2; ++e) {
                        const float2 u = make_float2(src[(2 * e) * DK], src[(2 * e + 1) * DK]);
                        S[e] = s == np ? u : __ffma2_rn(make_float2(gp, gp), S[e], u);
                    }
                }
            } else if (init && blockIdx.y == 0) {
                const StT* src = static_cast<const StT*>(p.pool) + (int64_t)slot * slot_elems + row;
#pragma unroll
                for (int e = 0; e < kLHalf; ++e) {
                    const float x = dvh + e < p.DV ? to_f32(src[(int64_t)e * DK]) : 0.f;
                    if (e & 1) S[e / 2].y = x; else S[e / 2].x = x;
                }
            }
            if (kState && blockIdx.y == 0) {
#pragma unroll
                for (int e = 0; e < kLHalf; ++e) wsp[e * DK] = (e & 1) ? S[e / 2].y : S[e / 2].x;
            }
        }
        auto put_state = [&]() {  // S in bf16, rows dk
            if (mine) {
#pragma unroll
                for (int c8 = 0; c8 < kLHalf / 8; ++c8) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) w[u] = bf16x2_bits(S[4 * c8 + u].x, S[4 * c8 + u].y);
                    *reinterpret_cast<uint4*>(sm + PL::SH_OFF + sw128(DK, lt, 4 * hf + c8)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(kSReady));
        };
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            if constexpr (!kState) {
                ok = c == 0 || warp_wait(kIFull, (uint32_t)(c - 1) & 1u);  // the last inter product has read S
                if (!ok) break;
                put_state();
            }
            ok = warp_wait(kUFull + (c & 1), (uint32_t)(c >> 1) & 1u);
            if (!ok) break;
            tc_fence_after();
            const int m = min(kLC, n - c * kLC);
            const float gm = pw[m];
            bool slow = false;
#pragma unroll
            for (int c0 = 0; c0 < kLHalf; c0 += 16) {
                float u[16];
                tmem_ld16(lane_base + u_col(c) + kLHalf * hf + c0, u);
                tmem_wait_ld();
                // A k that is not finite makes all of its row of the product so, whatever V is (0 too): one number tells.  Parts of an
                // infinity sum to NaN: the state that such tokens give is then formed from the tokens themselves.
                if (c0 == 0) slow = __any_sync(0xffffffffu, mine && (odd[c & 3] == c + 1 || !(fabsf(u[0]) <= FLT_MAX)));
                if (slow) break;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    S[c0 / 2 + e] = __ffma2_rn(make_float2(gm, gm), S[c0 / 2 + e], make_float2(u[2 * e], u[2 * e + 1]));
            }
            if (slow) {  // g^m S waits in the place of the product, so that the loop below has the registers
                const uint32_t at = lane_base + u_col(c) + kLHalf * hf;
#pragma unroll
                for (int c0 = 0; c0 < kLHalf; c0 += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(gm * ((e & 1) ? S[(c0 + e) / 2].y : S[(c0 + e) / 2].x));
                    tmem_st8(at + c0, w);
                }
                tmem_wait_st();
                add_tokens<DK>(p, place, pw, at, c, m);
#pragma unroll
                for (int c0 = 0; c0 < kLHalf; c0 += 16) {
                    float x[16];
                    tmem_ld16(at + c0, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) S[c0 / 2 + e] = make_float2(x[2 * e], x[2 * e + 1]);
                }
            }
            tc_fence_before();
            mbar_arrive(bar(kUFree + (c & 1)));
        }
        if (ok && mine) {
            if constexpr (kState) {
                float* dst = wsp + (int64_t)(blockIdx.y + 1) * (kLDv * DK);
#pragma unroll
                for (int e = 0; e < kLHalf; ++e) dst[e * DK] = (e & 1) ? S[e / 2].y : S[e / 2].x;
            } else if (last && out >= 0) {
                StT* dst = static_cast<StT*>(p.pool) + (int64_t)out * slot_elems + row;
#pragma unroll
                for (int e = 0; e < kLHalf; ++e) {
                    const float x = (e & 1) ? S[e / 2].y : S[e / 2].x;
                    if (dvh + e < p.DV) {
                        if constexpr (std::is_same<StT, float>::value)
                            dst[(int64_t)e * DK] = x;
                        else
                            dst[(int64_t)e * DK] = __float2bfloat16_rn(x);
                    }
                }
            }
        }
    } else if (warp < 24) {
        // ============ thread = token, half of the tile: V'; thread = row i, half of the tile: o ============
        const float gi = pw[lt + 1];
        auto write_o = [&](int c) -> bool {  // kOFull has been seen
            tc_fence_after();
            const int m = min(kLC, n - c * kLC);
            __nv_bfloat16* dst =
                static_cast<__nv_bfloat16*>(p.o) + ((int64_t)(tok0 + c * kLC + lt) * p.HV + h) * p.DV + dv0;
            const bool slow = odd[c & 3] == c + 1;  // then V is read once more
            // whole chunks go through shared memory and out by TMA: stored from here, 32 rows of 16 bytes an instruction, they took
            // 2000 cycles
            const bool staged = !slow && m == kLC;
            unsigned char* ot = sm + (PL::OWN ? PL::O_OFF : stage(c) + PL::V_OFF);
            if (PL::OWN && c > 0 && !warp_wait(kStFree, (uint32_t)(c - 1) & 1u)) return false;
#pragma unroll 1
            for (int c0 = kLHalf * hf; c0 < kLHalf * hf + kLHalf; c0 += 16) {
                float a[16], x[16];
                tmem_ld16(lane_base + kO1Col + c0, a);
                tmem_ld16(lane_base + kO2Col + c0, x);
                tmem_wait_ld();
                if (slow) {
                    // 0 times an infinity of a later token must not reach this row: its own tokens alone, one by one
#pragma unroll
                    for (int e = 0; e < 16; ++e) a[e] = 0.f;
#pragma unroll 1
                    for (int jw = 0; jw < kLC / 2; ++jw) {  // two weights a word of P
                        uint32_t pp;
                        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                                     : "=r"(pp)
                                     : "r"(lane_base + kScCol + (uint32_t)(c & 1) * 128 + (jw < 32 ? jw : jw + 32)));
                        tmem_wait_ld();
#pragma unroll 1
                        for (int jj = 0; jj < 2; ++jj) {
                            const int j = 2 * jw + jj;
                            const float wj = __uint_as_float(jj ? pp & 0xffff0000u : pp << 16);
                            if (j > lt || j >= m) continue;
#pragma unroll
                            for (int e = 0; e < 16; e += 8) {
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
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 y = __fmul2_rn(
                            make_float2(p.scale, p.scale),
                            __ffma2_rn(make_float2(gi, gi), make_float2(x[e + 2 * u], x[e + 2 * u + 1]),
                                       make_float2(a[e + 2 * u], a[e + 2 * u + 1])));
                        w[u] = bf16x2_bits(y.x, y.y);
                    }
                    if (staged)
                        *reinterpret_cast<uint4*>(ot + sw128(kLC, lt, (c0 + e) / 8)) = make_uint4(w[0], w[1], w[2], w[3]);
                    else if (lt < m && dv0 + c0 + e < p.DV)
                        *reinterpret_cast<uint4*>(dst + c0 + e) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            tc_fence_before();
            mbar_arrive(bar(kOFree));
            fence_proxy_async_smem();
            mbar_arrive(bar(kStaged + (c & 1)));
            return true;
        };
        // V' of a chunk and o of the one before, whichever is there first
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const int m = min(kLC, n - c * kLC);
            const uint32_t parity = (uint32_t)(c >> 1) & 1u;
            bool o_left = !kState && c > 0;
            const int before = kState ? c - 2 : c - 1;  // the chunk whose V' was where this one's goes
            for (uint32_t polls = 0; polls < kLPolls; ++polls) {  // what has not come by then is waited for below
                // V' goes over another chunk's, which the update has read then; of a partial chunk K's rows are cleared too
                bool there = mbar_test(bar(kVFull + (c & 1)), parity);
                if (before >= 0) there &= mbar_test(bar(kUFull + (before & 1)), (uint32_t)(before >> 1) & 1u);
                if (m < kLC) there &= mbar_test(bar(kQkFull + (c & 1)), parity);
                if (__all_sync(0xffffffffu, there)) break;
                if (o_left && __all_sync(0xffffffffu, mbar_test(bar(kOFull), (uint32_t)(c - 1) & 1u))) {
                    ok = write_o(c - 1);
                    o_left = false;
                    break;
                }
                __nanosleep(20);
                if (__any_sync(0xffffffffu, *fail != 0)) {
                    ok = false;
                    break;
                }
            }
            ok = ok && warp_wait(kVFull + (c & 1), parity) &&
                 (before < 0 || warp_wait(kUFull + (before & 1), (uint32_t)(before >> 1) & 1u)) &&
                 (m == kLC || warp_wait(kQkFull + (c & 1), parity));
            if (!ok) break;
            unsigned char* vt = sm + stage(c) + PL::V_OFF;
            const bool real = lt < m;
            const float f = real ? pw[m - 1 - lt] : 0.f;
            float2 probe = make_float2(0.f, 0.f);
            if (!real) {  // rows behind the prompt's last token belong to others, or to nobody
#pragma unroll
                for (int c8 = hf * DK / 16; c8 < (hf + 1) * DK / 16; ++c8)
                    *reinterpret_cast<uint4*>(sm + stage(c) + PL::K_OFF + sw128(kLC, lt, c8)) = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c8 = 4 * hf; c8 < 4 * hf + 4; ++c8) *reinterpret_cast<uint4*>(vt + sw128(kLC, lt, c8)) = make_uint4(0, 0, 0, 0);
            }
#pragma unroll 2
            for (int c8 = 4 * hf; c8 < 4 * hf + 4; ++c8) {
                const uint32_t at = sw128(kLC, lt, c8);
                const uint4 v4 = *reinterpret_cast<const uint4*>(vt + at);
                const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
                uint32_t w[NP][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float2 v2 = bf16x2_to_float2(vw[u]);
                    probe = __ffma2_rn(v2, make_float2(0.f, 0.f), probe);  // 0 unless one is not finite
                    float2 x = __fmul2_rn(make_float2(f, f), v2);
#pragma unroll
                    for (int e = 0; e < NP; ++e) w[e][u] = take_bf16(x);
                }
#pragma unroll
                for (int e = 0; e < NP; ++e)
                    *reinterpret_cast<uint4*>(sm + PL::vp(kState && (c & 1), e) + at) =
                        make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
            }
            if (!(probe.x == 0.f && probe.y == 0.f)) odd[c & 3] = c + 1;
            fence_proxy_async_smem();
            mbar_arrive(bar(kVReady + (c & 1)));
            if (kState) mbar_arrive(bar(kEmptyV + (c & 1)));
            if (o_left) {
                ok = warp_wait(kOFull, (uint32_t)(c - 1) & 1u) && write_o(c - 1);
                if (!ok) break;
            }
        }
        if (!kState && ok && nch > 0 && warp_wait(kOFull, (uint32_t)(nch - 1) & 1u)) write_o(nch - 1);
    } else if (tid == 3 * kLGroup) {
        // ============ tiles by TMA ============
#ifdef GDN_TEST_MISSING_COPY
        int qk = item > 0 || blockIdx.y > 0 ? min(nch, 2) : 0, v = qk;
#else
        int qk = min(nch, 2), v = qk;  // chunks asked for
#endif
        for (int c = qk; c < nch && qk > 0; ++c) {
            const uint32_t parity = (uint32_t)((c - 2) >> 1) & 1u;
            if (kState) {  // V is free first, else K and Q are
                if (!wait(kEmptyV + (c & 1), parity)) break;
                load_v(c);
                v = c + 1;
            }
            if (!wait(kEmptyQk + (c & 1), parity)) break;
            load_qk(c);
            qk = c + 1;
            if (!kState) {
                if (!wait(kEmptyV + (c & 1), parity)) break;
                load_v(c);
                v = c + 1;
            }
        }
        // copies in flight land before the CTA leaves
        for (int c = max(0, qk - 2); c < qk; ++c) mbar_wait_bounded(bar(kQkFull + (c & 1)), (uint32_t)(c >> 1) & 1u, kLPolls);
        for (int c = max(0, v - 2); c < v; ++c) mbar_wait_bounded(bar(kVFull + (c & 1)), (uint32_t)(c >> 1) & 1u, kLPolls);
    } else if (warp == 25) {
        // ============ products ============
        // The whole warp runs this code, so that descriptors stay in registers of the warp (from code of a single thread a product
        // took 100 cycles to issue, where it runs 32 to 64), and waits for up to three barriers at once, a lane for each.
        bool any = false, ok = true;
        const bool lead = elect_one();
        const uint32_t tm = __reduce_or_sync(0xffffffffu, tmem);
        constexpr uint32_t kBn = 1u << 16, kAm = 1u << 15;  // B N-major, A M-major
        constexpr uint32_t id64 = umma_idesc_bf16(128, kLDv);
        const int ln = tid & 31;
        auto all_over = [&](int b0, int c0, int b1, int c1, int b2, int c2) -> bool {  // phase c of barrier b, c1 and c2 < 0: none
            const bool one = ln == 1 && c1 >= 0, two = ln == 2 && c2 >= 0;
            return warp_wait(one ? b1 : two ? b2 : b0, (uint32_t)(one ? c1 : two ? c2 : c0) & 1u);
        };
        auto scores = [&](int c) {
            tc_fence_after();
            const uint32_t st = base + stage(c);
            if (lead) {
#pragma unroll 2
                for (int ks = 0; ks < DK / 16; ++ks) {
                    const uint32_t off = (uint32_t)(ks >> 2) * PL::BOX + (uint32_t)(ks & 3) * 32u;
                    umma_bf16(tm + kScCol + (uint32_t)(c & 1) * 128, umma_desc_sw128(st + PL::Q_OFF + off),
                              umma_desc_sw128(st + PL::K_OFF + off), umma_idesc_bf16(kLC, kLC), ks > 0 ? 1u : 0u);
                }
                umma_commit(bar(kScFull + (c & 1)));
            }
            any = true;
        };
        // a last, partial chunk's scores wait for its rows to be cleared
        auto whole = [&](int c) { return n - c * kLC >= kLC; };
        if (!kState && nch > 0) {
            ok = all_over(kQkFull, 0, kVReady, whole(0) ? -1 : 0, 0, -1);
            if (ok) scores(0);
        }
        for (int c = 0; c < nch && ok; ++c) {
            const uint32_t st = base + stage(c);
            // U: K^T V'.  The state waits for it alone.
            const int before = kState ? c - 2 : c - 1;
            ok = all_over(kVReady + (c & 1), c >> 1, kUFree + (before & 1), before >> 1, kQkFull + (c & 1), c >> 1);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
                for (int part = 0; part < NP; ++part)
#pragma unroll 2
                    for (int ks = 0; ks < kLC / 16; ++ks)
                        umma_bf16(tm + u_col(c), umma_desc_sw128_mn(st + PL::K_OFF + ks * 2048u, PL::BOX),
                                  umma_desc_sw128_mn(base + PL::vp(kState && (c & 1), part) + ks * 2048u, PL::BOX),
                                  id64 | kBn | kAm, part + ks > 0 ? 1u : 0u);
                umma_commit(bar(kUFull + (c & 1)));
                if (kState) {
                    umma_commit(bar(kEmptyQk + (c & 1)));
                }
            }
            any = true;
            if constexpr (!kState) {
                ok = all_over(kSReady, c, kOFree, c - 1, 0, -1);
                if (!ok) break;
                tc_fence_after();
                if (lead) {
#pragma unroll 2
                    for (int ks = 0; ks < DK / 16; ++ks) {
                        const uint32_t off = (uint32_t)(ks >> 2) * PL::BOX + (uint32_t)(ks & 3) * 32u;
                        umma_bf16(tm + kO2Col, umma_desc_sw128(st + PL::Q_OFF + off),
                                  umma_desc_sw128_mn(base + PL::SH_OFF + ks * 2048u, PL::BOX), id64 | kBn, ks > 0 ? 1u : 0u);
                    }
                    umma_commit(bar(kIFull));
                    umma_commit(bar(kEmptyQk + (c & 1)));  // scores, update and inter products have read K and Q
                }
                // The intra product and the next scores, which go over the P that the last chunk's intra product has read: in
                // this order where P is there (V is free for the next load earlier), else the scores first if their tiles are
                const int nx = c + 1;
                bool late = nx < nch;
                if (late && whole(nx) && !__all_sync(0xffffffffu, mbar_test(bar(kPReady + (c & 1)), (uint32_t)(c >> 1) & 1u)) &&
                    __all_sync(0xffffffffu, mbar_test(bar(kQkFull + (nx & 1)), (uint32_t)(nx >> 1) & 1u))) {
                    scores(nx);
                    late = false;
                }
                ok = all_over(kPReady + (c & 1), c >> 1, 0, -1, 0, -1);
                if (!ok) break;
                tc_fence_after();
                if (lead) {
#pragma unroll 2
                    for (int ks = 0; ks < kLC / 16; ++ks)
                        umma_bf16_ta(tm + kO1Col, tm + kScCol + (uint32_t)(c & 1) * 128 + (ks < 4 ? 8 * ks : 32 + 8 * ks),
                                     umma_desc_sw128_mn(st + PL::V_OFF + ks * 2048u, PL::BOX), id64 | kBn, ks > 0 ? 1u : 0u);
                    umma_commit(bar(kOFull));
                    if (PL::OWN) umma_commit(bar(kEmptyV + (c & 1)));
                }
                if (late) {
                    ok = all_over(kQkFull + (nx & 1), nx >> 1, kVReady + (nx & 1), whole(nx) ? -1 : nx >> 1, 0, -1);
                    if (ok) scores(nx);
                }
            }
        }
        if (any) {  // every product is complete before the tensor memory is released
            if (lead) umma_commit(bar(kDrain));
            for (uint32_t k = 0; k < kLPolls && !__all_sync(0xffffffffu, mbar_try_wait(bar(kDrain), 0u)); ++k) {}  // whatever has failed
        }
    } else if (tid == 3 * kLGroup + 64 && !kState) {
        // ============ o out ============
        for (int c = 0; c < nch; ++c) {
            if (!wait(kStaged + (c & 1), (uint32_t)(c >> 1) & 1u)) break;
            if (n - c * kLC >= kLC && odd[c & 3] != c + 1) {
                tma_store_3d(&maps.o, dv0, h, tok0 + c * kLC, base + (PL::OWN ? PL::O_OFF : stage(c) + PL::V_OFF));
                bulk_commit_group();
                bulk_wait_read_all();
            }
            mbar_arrive(bar(PL::OWN ? kStFree : kEmptyV + (c & 1)));
        }
        bulk_wait_all();
    } else if (tid == 3 * kLGroup + 96 && PL::OWN && !kState) {
        // ============ V read: by V' and the intra product (which arrives by itself), and where it is not finite once more ============
        for (int c = 0; c < nch; ++c) {
            const uint32_t parity = (uint32_t)(c >> 1) & 1u;
            if (!wait(kVReady + (c & 1), parity) || (odd[c & 3] == c + 1 && !wait(kStaged + (c & 1), parity))) break;
            mbar_arrive(bar(kEmptyV + (c & 1)));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *fail != 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, kLCols);
}

// Tokens of a piece (a multiple of the chunk), 0 where prompts stay whole.  Cutting reads K and V once more, so it must at
// least double the SMs at work.
int linear_split(int B, int N, int HV, int DV) {
    const int64_t items = (int64_t)B * HV * ((DV + kLDv - 1) / kLDv);
    if (items == 0 || N == 0) return 0;
    const int sms = sm_count();
    const int64_t times = (sms > 0 ? sms : 152) / items;  // pieces that fill the GPU once
    if (times < 2) return 0;
    const int64_t chunks = (N / B + (int64_t)kLC - 1) / kLC;
    const int64_t per = (chunks + times - 1) / times > 4 ? (chunks + times - 1) / times : 4;
    if (3 * per > 2 * chunks) return 0;  // prompts of less than a piece and a half on average
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
    using PL = LinearPlan<DK, std::is_same<StT, float>::value ? 3 : 2>;
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
    const int pieces = piece > 0 ? (int)(((int64_t)p.N + piece - 1) / piece) : 1;
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
    return ((int64_t)N + piece - 1) / piece * B * HV * ((DV + kLDv - 1) / kLDv) * kLDv * DK * 4;
}

bool launch_linear_prefill(const LinearParams& p, bool qkv_bf16, bool state_bf16, float* ws, cudaStream_t s, cudaError_t& err) {
    const int64_t items = (int64_t)p.B * p.HV * ((p.DV + kLDv - 1) / kLDv);
    if ((p.DK != 64 && p.DK != 128) || !qkv_bf16 || !p.out_bf16 || !p.v_vec || (reinterpret_cast<uintptr_t>(p.o) & 15u) != 0 ||
        p.N == 0 || items > 0x7fffffff)
        return false;
    LinearMaps m;
    std::memset(&m, 0, sizeof m);
    if (!encode_rows(&m.q, p.q, p.DK, p.HK, p.N) || !encode_rows(&m.k, p.k, p.DK, p.HK, p.N) ||
        !encode_rows(&m.v, p.v, p.DV, p.HV, p.N) || !encode_rows(&m.o, p.o, p.DV, p.HV, p.N))
        return false;
    if (p.DK == 64)
        err = state_bf16 ? launch_dk<64, __nv_bfloat16>(p, m, ws, s) : launch_dk<64, float>(p, m, ws, s);
    else
        err = state_bf16 ? launch_dk<128, __nv_bfloat16>(p, m, ws, s) : launch_dk<128, float>(p, m, ws, s);
    return true;
}

}  // namespace gdn
