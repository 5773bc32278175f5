// gdn_linear.cuh -- linear attention with a fixed decay for each head, a few tokens at a time (sm_103a):
//     S_t = g S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   g = exp(log_decay[h])
// for decode, verify, commit and the prompts that the tensor-core kernel does not take.  bf16 tokens of a step are products on mma.sync (the second
// kernel below, and the streaming one for many lanes); fp32 tokens, DK 16, DK 256 with fp32 states and prompts are the first kernel's, on the CUDA cores.
//
// Over n tokens from a state S_0 the recurrence unrolls to
//     o_t = scale (g^{t+1} S_0 q_t + sum_{j <= t} w_tj v_j),   w_tj = g^{t-j} (k_j . q_t)
//     S_n = g^n S_0 + sum_j g^{n-1-j} v_j k_j^T
// so a row of the state meets every token in one dot product, and takes one multiply-add a token when it is kept at all:
// a verify that keeps nothing does a third of the work of the step-by-step form.  Only powers g^e with e >= 0 appear, so no
// decay overflows, and g^0 is 1 for g = 0 too.  A verify that stores the state after every token goes step by step.
//
// In the first kernel a CTA of 4 warps holds RPC rows of one (lane, head) in fp32 registers (the lane layout of Split: 8 columns of RL rows a
// lane) and takes the tokens in chunks of up to 16 from shared memory.  Bytes bound a token or two (decode of 128 lanes, D 128, fp32 tokens and
// states: 118 us, 4.6 TB/s); more tokens are bound by their dot products and shared-memory reads (verify of 128 lanes x 8 with bf16 states 153 us,
// five times its bytes; prompts of 4 x 2048, HV 32, D 128: 2440 us with fp32 tokens, 2330 with DV 100, 6160 with DK 256).
#pragma once

#include <type_traits>

#include "gdn_common.cuh"

namespace gdn {

constexpr int kLinChunk = 16;

// shared memory, in floats, for chunks of CT tokens: q, k [CT][DK], v [CT][RPC], w [CT][CT], g^0 .. g^CT
template <int DK>
__host__ __device__ constexpr int linear_smem_floats(int CT) {
    return 2 * CT * DK + CT * Split<DK>::RPC + CT * CT + CT + 1;
}

template <int DK, typename InT, typename StT, bool kKept>
__global__ void __launch_bounds__(Split<DK>::THREADS, Split<DK>::MIN_CTAS_PER_SM) gdn_linear_kernel(const LinearParams p,
                                                                                                   const int CT) {
    using SP = Split<DK>;
    using QK = Slice8<InT>;
    constexpr int RL = SP::RL, P = SP::P, NT = SP::THREADS, RPC = SP::RPC;
    extern __shared__ float4 smem4[];
    float* qs = reinterpret_cast<float*>(smem4);
    float* ks = qs + CT * DK;
    float* vs = ks + CT * DK;
    float* ws = vs + CT * RPC;
    float* pw = ws + CT * CT;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pc = lane % P, rg = lane / P;
    const int h = blockIdx.y, b = blockIdx.z, row0 = blockIdx.x * RPC, hk = h / (p.HV / p.HK);
    const int slot = p.indices[b];
    if (slot == -1) return;
    int out = p.write ? (p.out_indices != nullptr ? p.out_indices[b] : slot) : -1;
    if (slot < -1 || slot >= p.num_slots || out < -1 || out >= p.num_slots) {
        if (tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
        return;
    }
    int64_t tok0;
    int n;
    bool init = true;
    if (p.cu_seqlens != nullptr) {
        const int lo = p.cu_seqlens[b], hi = p.cu_seqlens[b + 1];
        if (lo < 0 || hi < lo || hi > p.N) {
            if (tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_SEQLEN);
            return;
        }
        tok0 = lo;
        n = hi - lo;
        init = p.has_init == nullptr || p.has_init[b] != 0;
    } else {
        tok0 = (int64_t)b * p.T;
        n = p.steps != nullptr ? p.steps[b] : p.T;
        if (n < 0 || n > p.T) {
            if (tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_ACCEPT_LEN);
            return;
        }
    }
    if (n == 0 && (out < 0 || out == slot)) return;  // nothing to do: the slot stays as it is

    const LaneRows<DK> lr(warp, rg, pc);
    const StT* src = static_cast<const StT*>(p.pool) + (((int64_t)slot * p.HV + h) * p.DV + row0) * DK;
    uint4 raw[RL][Slice8<StT>::NC];
#pragma unroll
    for (int i = 0; i < RL; ++i) {
#pragma unroll
        for (int c = 0; c < Slice8<StT>::NC; ++c) raw[i][c] = make_uint4(0, 0, 0, 0);
        if (init && row0 + lr.row[i] < p.DV) Slice8<StT>::load_global(src + (int64_t)lr.row[i] * DK + 8 * pc, raw[i]);
    }
    const float ld = p.log_decay[h];
    if (tid <= CT) pw[tid] = decay_power(ld, tid);
    float2 S[RL][4];
    const InT* qp = static_cast<const InT*>(p.q);
    const InT* kp = static_cast<const InT*>(p.k);
    const InT* vp = static_cast<const InT*>(p.v);

    // the complete dot product of this lane's own row with the 8-column pieces x2 of all lanes of the row group
    auto row_dots = [&](const float2 (&x2)[4]) {
        float c[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __ffma2_rn(S[i][e], x2[e], acc);
            c[i] = acc.x + acc.y;
        }
#pragma unroll
        for (int l = 0; l < SP::LOG_RL; ++l)
#pragma unroll
            for (int j = 0; j < (RL >> (l + 1)); ++j)
                c[j] += __shfl_xor_sync(0xffffffffu, c[j + (RL >> (l + 1))], P >> (l + 1));
#pragma unroll
        for (int m = P >> (SP::LOG_RL + 1); m >= 1; m >>= 1) c[0] += __shfl_xor_sync(0xffffffffu, c[0], m);
        return c[0];
    };
    auto piece = [&](const float* row, float2 (&x2)[4]) {  // columns 8 pc .. 8 pc + 7 of a q or k row in shared memory
        const float4 a = *reinterpret_cast<const float4*>(row + 4 * pc);
        const float4 d = *reinterpret_cast<const float4*>(row + DK / 2 + 4 * pc);
        x2[0] = make_float2(a.x, a.y);
        x2[1] = make_float2(a.z, a.w);
        x2[2] = make_float2(d.x, d.y);
        x2[3] = make_float2(d.z, d.w);
    };
    const bool owner = pc == SP::owner_p(lr.code) && row0 + lr.own_row < p.DV;
    auto store_o = [&](int64_t t, float x) {
        const int64_t at = ((tok0 + t) * p.HV + h) * p.DV + row0 + lr.own_row;
        if (!owner) return;
        if (p.out_bf16)
            static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(p.scale * x);
        else
            static_cast<float*>(p.o)[at] = p.scale * x;
    };

    bool unpacked = false;
    for (unsigned c0 = 0; c0 < (unsigned)n; c0 += CT) {  // unsigned: n may be near 2^31
        const int m = min(CT, n - (int)c0);
        if (c0 > 0) __syncthreads();  // the last chunk's tokens are no longer read
        // tokens into shared memory: P threads a q or k row
        for (int j = tid / P; j < m; j += NT / P) {
            const int64_t off = ((tok0 + c0 + j) * p.HK + hk) * DK + 8 * (tid % P);
            uint4 r[QK::NC];
            float2 x2[4];
            float* dst = ks + j * DK + 4 * (tid % P);
            QK::load_global(kp + off, r);
            QK::unpack(r, x2);
            *reinterpret_cast<float4*>(dst) = make_float4(x2[0].x, x2[0].y, x2[1].x, x2[1].y);
            *reinterpret_cast<float4*>(dst + DK / 2) = make_float4(x2[2].x, x2[2].y, x2[3].x, x2[3].y);
            if (qp != nullptr) {
                dst = qs + j * DK + 4 * (tid % P);
                QK::load_global(qp + off, r);
                QK::unpack(r, x2);
                *reinterpret_cast<float4*>(dst) = make_float4(x2[0].x, x2[0].y, x2[1].x, x2[1].y);
                *reinterpret_cast<float4*>(dst + DK / 2) = make_float4(x2[2].x, x2[2].y, x2[3].x, x2[3].y);
            }
        }
        for (int e = tid; e < m * RPC; e += NT) {
            const int j = e / RPC, r = e % RPC;
            vs[e] = row0 + r < p.DV ? to_f32(vp[((tok0 + c0 + j) * p.HV + h) * p.DV + row0 + r]) : 0.f;
        }
        __syncthreads();
        if (!kKept && qp != nullptr) {  // w_tj, P lanes a pair
            for (int e = tid / P; e < m * m; e += NT / P) {
                const int t = e / m, j = e % m;
                if (j > t) continue;
                // P lanes of one warp share e, so they take the branch together
                float2 a2[4], b2[4];
                piece(ks + j * DK, a2);
                piece(qs + t * DK, b2);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < 4; ++x) acc = __ffma2_rn(a2[x], b2[x], acc);
                float d = acc.x + acc.y;
                const unsigned mask = P == 32 ? 0xffffffffu : ((1u << (P & 31)) - 1u) << (lane & ~(P - 1));
#pragma unroll
                for (int x = 1; x < P; x <<= 1) d += __shfl_xor_sync(mask, d, x);
                if (pc == 0) ws[t * CT + j] = pw[t - j] * d;
            }
            __syncthreads();
        }
        if (!unpacked) {
            unpacked = true;
#pragma unroll
            for (int i = 0; i < RL; ++i) Slice8<StT>::unpack(raw[i], S[i]);
        }
        if constexpr (kKept) {
            const float g = pw[1];
            for (int t = 0; t < m; ++t) {
                float2 k2[4], q2[4];
                piece(ks + t * DK, k2);
                piece(qs + t * DK, q2);
#pragma unroll
                for (int i = 0; i < RL; ++i) {
                    const float d = vs[t * RPC + lr.row[i]];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[i][e] = __ffma2_rn(make_float2(d, d), k2[e], __fmul2_rn(make_float2(g, g), S[i][e]));
                    if (row0 + lr.row[i] < p.DV)
                        Slice8<StT>::template store_global<true>(
                            static_cast<StT*>(p.cache) +
                                ((((int64_t)b * p.T + t) * p.HV + h) * p.DV + row0 + lr.row[i]) * DK + 8 * pc,
                            S[i]);
                }
                store_o(t, row_dots(q2));
            }
        } else {
            if (qp != nullptr) {
                for (int t = 0; t < m; ++t) {
                    float2 q2[4];
                    piece(qs + t * DK, q2);
                    float x = pw[t + 1] * row_dots(q2);
                    for (int j = 0; j <= t; ++j) x = fmaf(ws[t * CT + j], vs[j * RPC + lr.own_row], x);
                    store_o(c0 + t, x);
                }
            }
            if (out >= 0 || c0 + CT < (unsigned)n) {
                const float gm = pw[m];
#pragma unroll
                for (int i = 0; i < RL; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][e] = __fmul2_rn(make_float2(gm, gm), S[i][e]);
                for (int j = 0; j < m; ++j) {
                    float2 k2[4];
                    piece(ks + j * DK, k2);
                    const float f = pw[m - 1 - j];
#pragma unroll
                    for (int i = 0; i < RL; ++i) {
                        const float d = f * vs[j * RPC + lr.row[i]];
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[i][e] = __ffma2_rn(make_float2(d, d), k2[e], S[i][e]);
                    }
                }
            }
        }
    }
    if (out < 0) return;
    if (!unpacked)  // no tokens: the state as it was read
#pragma unroll
        for (int i = 0; i < RL; ++i) Slice8<StT>::unpack(raw[i], S[i]);
    StT* dst = static_cast<StT*>(p.pool) + (((int64_t)out * p.HV + h) * p.DV + row0) * DK;
#pragma unroll
    for (int i = 0; i < RL; ++i)
        if (row0 + lr.row[i] < p.DV)
            Slice8<StT>::template store_global<false>(dst + (int64_t)lr.row[i] * DK + 8 * pc, S[i]);
}

// ---- bf16 tokens: products on mma.sync ------------------------------------------------------------------------
// The same unrolled form, a warp for 16 rows of a (lane, head) and no barrier in the way of the loads.  S_0 q_t, q_t . k_j and
// the sum over j are products of small matrices, which mma.sync (m16n8k16, bf16 with fp32 sums) does with a few
// instructions where the lane layout above needs a dot product a row and token: 8 tokens of 16 rows of 128 are 8 + 8 + 3
// instructions.  (tcgen05 would want 64 rows a tile and a trip through shared memory for work that bytes bound anyway.)
//   * Lane (g, t) = (lane / 4, lane % 4) holds rows 2g and 2g + 1, and of each 32 columns the 8 from 8t: one 16-byte load of bf16.
//     A dot product does not mind the order of its terms, so those 8 serve as the columns that two products expect.
//   * Factors that are not bf16 go in as three bf16 parts (24 bits, what fp32 holds): w_tj, and the elements of fp32 states.
//   * A token's q as the product's column for S q is, register by register, its row for q . k.
// A value that is not finite would reach earlier tokens as 0 times it: then the sum over j is formed term by term.
// Measured (HK 16, HV 32, D 128, in graph replays): decode of 64 lanes with fp32 states 46.6 us (5.8 TB/s; the lane layout above: 63), verify of
// 128 x 4 with states kept 100.5 (6.8 TB/s; 137), commit of 128 x 8 with fp32 states 92 (5.9 TB/s); 9 to 16 tokens of 256 lanes, bf16 states: verify
// 94 to 114, commit 121 to 137, decode 211 to 300, two to three times their bytes (loads behind the slot, stores behind the products).  Verify and
// commit of many lanes and up to 8 tokens wait for loads here and are the streaming kernel's (gdn_linear_stream.cuh); two blocks of rows a
// warp measured the same or slower (fewer warps).
enum { kLinVerify, kLinDecode, kLinKept, kLinCommit };
constexpr int kLinWarps = 4;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x, y) as three pairs of bf16
__device__ __forceinline__ void three_parts(float x, float y, uint32_t (&w)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        w[i] = Chunk<__nv_bfloat16>::pack2(x, y);
        x -= __uint_as_float(w[i] << 16);
        y -= __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <typename StT>
struct RowPiece;  // 8 columns of a row
template <>
struct RowPiece<__nv_bfloat16> {
    uint4 r;
    static constexpr int PARTS = 1;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = ld_state16(p); }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    // columns 4s .. 4s + 3 as the operand words of product s
    __device__ __forceinline__ void words(int s, uint32_t (&lo)[1], uint32_t (&hi)[1]) const {
        lo[0] = s == 0 ? r.x : r.z;
        hi[0] = s == 0 ? r.y : r.w;
    }
    __device__ __forceinline__ void unpack(float2 (&x)[4]) const {
        const uint4 a[1] = {r};
        Slice8<__nv_bfloat16>::unpack(a, x);
    }
};
template <>
struct RowPiece<float> {
    float4 a, b;
    static constexpr int PARTS = 3;
    __device__ __forceinline__ void load(const float* p) {
        const uint4 u = ld_state16(p), v = ld_state16(p + 4);
        a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
        b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void words(int s, uint32_t (&lo)[3], uint32_t (&hi)[3]) const {
        const float4 f = s == 0 ? a : b;
        three_parts(f.x, f.y, lo);
        three_parts(f.z, f.w, hi);
    }
    __device__ __forceinline__ void unpack(float2 (&x)[4]) const {
        x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w), x[2] = make_float2(b.x, b.y), x[3] = make_float2(b.z, b.w);
    }
};

__device__ __forceinline__ uint32_t word_of(const uint4& r, int i) { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }

// shared memory in bytes: k of the tokens in fp32 [T][DK] (where the state is updated), v words [warps][T][8]
template <int DK>
constexpr int linear_mma_smem(int T, bool update) {
    return (update ? T * DK * 4 : 0) + kLinWarps * T * 32;
}

// NTI: tokens / 8, rounded up.  CTAs an SM: as many as registers hold without spills to speak of.  bf16 states with DK 128 and outputs spilled
// 48 to 144 bytes with one more: us in graph replays then / now, 256 lanes of 16 tokens verify 155 / 114, decode 311 / 300, 128 lanes of 4 with
// states kept 107 / 100.5, decode of one lane 4.0 / 3.6; the commit, which does not spill, has it (16 tokens 137 / 147).  fp32 states with DK 64
// spill 4 to 16 bytes: one CTA less takes 81 instead of 94 for 256 lanes of 16 tokens, but 91.7 instead of 87.9 for their decode.
template <int DK, typename StT, int NTI, int kMode>
__global__ void __launch_bounds__(32 * kLinWarps, (sizeof(StT) * DK > 256 ? 4 : 6) - (NTI == 2) - (DK == 256) - (kMode != kLinCommit && sizeof(StT) == 2 && DK == 128)) gdn_linear_mma_kernel(const LinearParams p) {
    constexpr int NP = DK / 32;
    constexpr bool kOut = kMode != kLinCommit, kUpdate = kMode != kLinVerify;
    extern __shared__ float4 smem4[];
    float* ks = reinterpret_cast<float*>(smem4);
    const int T = p.T;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    uint32_t* vw = reinterpret_cast<uint32_t*>(ks + (kUpdate ? T * DK : 0)) + warp * T * 8;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (p.HV / p.HK);
    const int row = (blockIdx.x * kLinWarps + warp) * 16 + 2 * g;  // and row + 1
    const bool live0 = row < p.DV, live1 = row + 1 < p.DV;
    using bf16 = __nv_bfloat16;
    const bf16* kp = static_cast<const bf16*>(p.k) + ((int64_t)b * T * p.HK + hk) * DK;
    const bf16* qp = static_cast<const bf16*>(p.q) + ((int64_t)b * T * p.HK + hk) * DK;
    const bf16* vp = static_cast<const bf16*>(p.v) + ((int64_t)b * T * p.HV + h) * p.DV + row;
    const int64_t kstep = (int64_t)p.HK * DK, vstep = (int64_t)p.HV * p.DV;

    // what does not depend on the slot is asked for first
    const int slot = p.indices[b];
    int out = kMode == kLinDecode || kMode == kLinCommit ? (p.out_indices != nullptr ? p.out_indices[b] : slot) : -1;
    int n = T;
    if (kMode == kLinCommit) n = p.steps[b];
    uint4 qf[NTI][NP], kf[NTI][NP];
    if constexpr (kOut) {
#pragma unroll
        for (int i = 0; i < NTI; ++i)
#pragma unroll
            for (int c = 0; c < NP; ++c) {
                qf[i][c] = kf[i][c] = make_uint4(0, 0, 0, 0);
                if (8 * i + g < T) {
                    qf[i][c] = *reinterpret_cast<const uint4*>(qp + (8 * i + g) * kstep + 32 * c + 8 * t4);
                    kf[i][c] = *reinterpret_cast<const uint4*>(kp + (8 * i + g) * kstep + 32 * c + 8 * t4);
                }
            }
    }
    const float ld = p.log_decay[h];
    if (slot == -1) return;  // the whole CTA
    if (slot < -1 || slot >= p.num_slots || out < -1 || out >= p.num_slots) {
        if (tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_INDEX);
        return;
    }
    if (kMode == kLinCommit) {
        if (n < 0 || n > T) {
            if (tid == 0 && p.err != nullptr) atomicOr(p.err, GDN_ERRBIT_ACCEPT_LEN);
            return;
        }
        if (out < 0 || (n == 0 && out == slot)) return;  // nothing to write
    }
    RowPiece<StT> S[2][NP];
    {
        const StT* src = static_cast<const StT*>(p.pool) + (((int64_t)slot * p.HV + h) * p.DV + row) * DK + 8 * t4;
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            S[0][c].zero();
            S[1][c].zero();
            if (live0) S[0][c].load(src + 32 * c);
            if (live1) S[1][c].load(src + DK + 32 * c);
        }
    }
    // v of the warp's rows: words (row, row + 1) a token
    bool odd = false;
    for (int e = lane; e < n * 8; e += 32) {
        const int j = e >> 3, r = 2 * (e & 7) - 2 * g;  // relative to vp's row
        uint32_t w = 0;
        if (p.v_pair) {
            if (row + r < p.DV) w = *reinterpret_cast<const uint32_t*>(vp + j * vstep + r);
        } else {
            if (row + r < p.DV) w = *reinterpret_cast<const uint16_t*>(vp + j * vstep + r);
            if (row + r + 1 < p.DV) w |= (uint32_t) * reinterpret_cast<const uint16_t*>(vp + j * vstep + r + 1) << 16;
        }
        vw[e] = w;
        odd |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    }
    if constexpr (kUpdate) {
        for (int e = tid; e < n * (DK / 8); e += 32 * kLinWarps) {
            const int j = e / (DK / 8), c = e % (DK / 8);
            const uint4 r[1] = {*reinterpret_cast<const uint4*>(kp + j * kstep + 8 * c)};
            float2 x[4];
            Slice8<bf16>::unpack(r, x);
            float4* dst = reinterpret_cast<float4*>(ks + j * DK + 8 * c);
            dst[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
            dst[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
        }
        __syncthreads();
    } else {
        __syncwarp();
    }
    const float pw = decay_power(ld, lane);  // lane e: g^e (up to 16)
    auto power = [&](int e) { return __shfl_sync(0xffffffffu, pw, e & 31); };

    if constexpr (kOut) {
        odd = __any_sync(0xffffffffu, odd);
        float w[NTI][4];  // of tokens t = g (0, 1), g + 8 (2, 3) and j = 8 i + 2 t4, + 1
#pragma unroll
        for (int i = 0; i < NTI; ++i) {
            w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0.f;
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    mma_bf16(w[i], word_of(qf[0][c], 2 * s), NTI == 2 ? word_of(qf[NTI - 1][c], 2 * s) : 0u,
                             word_of(qf[0][c], 2 * s + 1), NTI == 2 ? word_of(qf[NTI - 1][c], 2 * s + 1) : 0u,
                             word_of(kf[i][c], 2 * s), word_of(kf[i][c], 2 * s + 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = g + (e & 2) * 4, j = 8 * i + 2 * t4 + (e & 1);
                const float f = power(t - j);
                w[i][e] = j <= t ? f * w[i][e] : 0.f;
            }
        }
        float sum[NTI][4];  // sum over j: rows row, row + 1 (0, 2 / 1, 3) and tokens 8 i + 2 t4, + 1
#pragma unroll
        for (int i = 0; i < NTI; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.f;
        if (!odd) {
            uint32_t va[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < NTI; ++i) {
                const int j = 8 * i + 2 * t4;
                const uint32_t x = j < n ? vw[j * 8 + g] : 0u, y = j + 1 < n ? vw[(j + 1) * 8 + g] : 0u;
                va[2 * i] = __byte_perm(x, y, 0x5410);
                va[2 * i + 1] = __byte_perm(x, y, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < NTI; ++i) {
                uint32_t b0[3], b1[3] = {0u, 0u, 0u};
                three_parts(w[0][2 * i], w[0][2 * i + 1], b0);
                if constexpr (NTI == 2) three_parts(w[NTI - 1][2 * i], w[NTI - 1][2 * i + 1], b1);
#pragma unroll
                for (int e = 0; e < 3; ++e) mma_bf16(sum[i], va[0], va[1], va[2], va[3], b0[e], b1[e]);
            }
        } else {
            for (int j = 0; j < n; ++j) {
                const uint32_t v2 = vw[j * 8 + g];
                const float v0 = __uint_as_float(v2 << 16), v1 = __uint_as_float(v2 & 0xffff0000u);
#pragma unroll
                for (int i = 0; i < NTI; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 8 * i + 2 * t4 + e, src = (t & 7) * 4 + (j & 7) / 2;
                        float x = 0.f;  // w_tj, from the lane that has it
#pragma unroll
                        for (int jt = 0; jt < NTI; ++jt) {
                            const float lo = __shfl_sync(0xffffffffu, w[jt][2 * i], src);
                            const float hi = __shfl_sync(0xffffffffu, w[jt][2 * i + 1], src);
                            if (jt == j / 8) x = (j & 1) ? hi : lo;
                        }
                        if (j <= t) {
                            sum[i][e] = fmaf(x, v0, sum[i][e]);
                            sum[i][2 + e] = fmaf(x, v1, sum[i][2 + e]);
                        }
                    }
            }
        }
        float dot[NTI][4];
#pragma unroll
        for (int i = 0; i < NTI; ++i) dot[i][0] = dot[i][1] = dot[i][2] = dot[i][3] = 0.f;
#pragma unroll
        for (int c = 0; c < NP; ++c)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                constexpr int NW = RowPiece<StT>::PARTS;
                uint32_t a0[NW], a1[NW], a2[NW], a3[NW];
                S[0][c].words(s, a0, a2);
                S[1][c].words(s, a1, a3);
#pragma unroll
                for (int e = 0; e < NW; ++e)
#pragma unroll
                    for (int i = 0; i < NTI; ++i)
                        mma_bf16(dot[i], a0[e], a1[e], a2[e], a3[e], word_of(qf[i][c], 2 * s), word_of(qf[i][c], 2 * s + 1));
            }
#pragma unroll
        for (int i = 0; i < NTI; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 8 * i + 2 * t4 + e;
                const float f = power(t + 1);
                const float x = p.scale * fmaf(f, dot[i][e], sum[i][e]), y = p.scale * fmaf(f, dot[i][2 + e], sum[i][2 + e]);
                if (t >= n || !live0) continue;
                const int64_t at = (((int64_t)b * T + t) * p.HV + h) * p.DV + row;
                if (p.out_bf16) {
                    bf16* dst = static_cast<bf16*>(p.o) + at;
                    if (p.o_pair)
                        *reinterpret_cast<uint32_t*>(dst) = Chunk<bf16>::pack2(x, y);
                    else {
                        dst[0] = __float2bfloat16_rn(x);
                        if (live1) dst[1] = __float2bfloat16_rn(y);
                    }
                } else {
                    float* dst = static_cast<float*>(p.o) + at;
                    dst[0] = x;
                    if (live1) dst[1] = y;
                }
            }
    }
    if constexpr (kUpdate) {
        if (kMode != kLinKept && out < 0) return;
        StT* dst = kMode == kLinKept
                       ? static_cast<StT*>(p.cache) + (((int64_t)b * T * p.HV + h) * p.DV + row) * DK + 8 * t4
                       : static_cast<StT*>(p.pool) + (((int64_t)out * p.HV + h) * p.DV + row) * DK + 8 * t4;
        const int64_t tstep = (int64_t)p.HV * p.DV * DK;
        const float g1 = power(1), gn = power(n);
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            float2 x[2][4];
            S[0][c].unpack(x[0]);
            S[1][c].unpack(x[1]);
            if (kMode != kLinKept)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[0][e] = __fmul2_rn(make_float2(gn, gn), x[0][e]);
                    x[1][e] = __fmul2_rn(make_float2(gn, gn), x[1][e]);
                }
            for (int j = 0; j < n; ++j) {
                const float4* kr = reinterpret_cast<const float4*>(ks + j * DK + 32 * c + 8 * t4);
                const float4 k0 = kr[0], k1 = kr[1];
                const float2 k2[4] = {make_float2(k0.x, k0.y), make_float2(k0.z, k0.w), make_float2(k1.x, k1.y),
                                      make_float2(k1.z, k1.w)};
                const uint32_t v2 = vw[j * 8 + g];
                float v0 = __uint_as_float(v2 << 16), v1 = __uint_as_float(v2 & 0xffff0000u);
                if (kMode == kLinKept) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[0][e] = __ffma2_rn(make_float2(v0, v0), k2[e], __fmul2_rn(make_float2(g1, g1), x[0][e]));
                        x[1][e] = __ffma2_rn(make_float2(v1, v1), k2[e], __fmul2_rn(make_float2(g1, g1), x[1][e]));
                    }
                    if (live0) Slice8<StT>::template store_global<true>(dst + j * tstep + 32 * c, x[0]);
                    if (live1) Slice8<StT>::template store_global<true>(dst + j * tstep + DK + 32 * c, x[1]);
                } else {
                    const float f = power(n - 1 - j);
                    v0 *= f;
                    v1 *= f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[0][e] = __ffma2_rn(make_float2(v0, v0), k2[e], x[0][e]);
                        x[1][e] = __ffma2_rn(make_float2(v1, v1), k2[e], x[1][e]);
                    }
                }
            }
            if (kMode != kLinKept) {
                if (live0) Slice8<StT>::template store_global<false>(dst + 32 * c, x[0]);
                if (live1) Slice8<StT>::template store_global<false>(dst + DK + 32 * c, x[1]);
            }
        }
    }
}

template <int DK, typename StT, int NTI>
cudaError_t launch_linear_mma(const LinearParams& p, cudaStream_t s) {
    const dim3 grid((p.DV + 16 * kLinWarps - 1) / (16 * kLinWarps), p.HV, p.B);
    const bool update = p.write || p.cache != nullptr;
    const size_t smem = linear_mma_smem<DK>(p.T, update);
    static_assert(linear_mma_smem<DK>(8 * NTI, true) <= 48 * 1024, "fits the default shared memory");
    if (p.q == nullptr)
        gdn_linear_mma_kernel<DK, StT, 1, kLinCommit><<<grid, 32 * kLinWarps, smem, s>>>(p);
    else if (p.cache != nullptr)
        gdn_linear_mma_kernel<DK, StT, NTI, kLinKept><<<grid, 32 * kLinWarps, smem, s>>>(p);
    else if (p.write)
        gdn_linear_mma_kernel<DK, StT, NTI, kLinDecode><<<grid, 32 * kLinWarps, smem, s>>>(p);
    else
        gdn_linear_mma_kernel<DK, StT, NTI, kLinVerify><<<grid, 32 * kLinWarps, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn

#include "gdn_linear_stream.cuh"

namespace gdn {

template <int DK, typename InT, typename StT>
cudaError_t launch_linear_dk(const LinearParams& p, cudaStream_t s) {
    // bf16 tokens of a step, where a warp's 16 rows fit its registers
    if constexpr (std::is_same<InT, __nv_bfloat16>::value && DK >= 32 && DK * sizeof(StT) <= 512) {
        cudaError_t e;
        if (p.cu_seqlens == nullptr && try_linear_stream<DK, StT>(p, s, e)) return e;
        if (p.cu_seqlens == nullptr) return p.T <= 8 ? launch_linear_mma<DK, StT, 1>(p, s) : launch_linear_mma<DK, StT, 2>(p, s);
    }
    using SP = Split<DK>;
    static_assert(kLinChunk >= GDN_MAX_T, "a step is one chunk");
    const int CT = p.cu_seqlens != nullptr ? kLinChunk : p.T;
    const size_t smem = sizeof(float) * linear_smem_floats<DK>(CT);
    static_assert(sizeof(float) * linear_smem_floats<DK>(kLinChunk) <= 48 * 1024, "fits the default shared memory");
    const dim3 grid((p.DV + SP::RPC - 1) / SP::RPC, p.HV, p.B);
    if (p.cache != nullptr)
        gdn_linear_kernel<DK, InT, StT, true><<<grid, SP::THREADS, smem, s>>>(p, CT);
    else
        gdn_linear_kernel<DK, InT, StT, false><<<grid, SP::THREADS, smem, s>>>(p, CT);
    return cudaGetLastError();
}

template <typename StT>
cudaError_t launch_linear(const LinearParams& p, bool qkv_bf16, cudaStream_t s) {
    switch (p.DK) {
    case 16: return qkv_bf16 ? launch_linear_dk<16, __nv_bfloat16, StT>(p, s) : launch_linear_dk<16, float, StT>(p, s);
    case 32: return qkv_bf16 ? launch_linear_dk<32, __nv_bfloat16, StT>(p, s) : launch_linear_dk<32, float, StT>(p, s);
    case 64: return qkv_bf16 ? launch_linear_dk<64, __nv_bfloat16, StT>(p, s) : launch_linear_dk<64, float, StT>(p, s);
    case 128: return qkv_bf16 ? launch_linear_dk<128, __nv_bfloat16, StT>(p, s) : launch_linear_dk<128, float, StT>(p, s);
    case 256: return qkv_bf16 ? launch_linear_dk<256, __nv_bfloat16, StT>(p, s) : launch_linear_dk<256, float, StT>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gdn
