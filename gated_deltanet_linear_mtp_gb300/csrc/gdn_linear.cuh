// gdn_linear.cuh -- linear attention with a fixed decay for each head, a few tokens at a time on the CUDA cores (sm_103a):
//     S_t = g S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   g = exp(log_decay[h])
// for decode, verify, commit and the prompts that the tensor-core kernel does not take.
//
// Over n tokens from a state S_0 the recurrence unrolls to
//     o_t = scale (g^{t+1} S_0 q_t + sum_{j <= t} w_tj v_j),   w_tj = g^{t-j} (k_j . q_t)
//     S_n = g^n S_0 + sum_j g^{n-1-j} v_j k_j^T
// so a row of the state meets every token in one dot product, and takes one multiply-add a token when it is kept at all:
// a verify that keeps nothing does a third of the work of the step-by-step form.  Only powers g^e with e >= 0 appear, so no
// decay overflows, and g^0 is 1 for g = 0 too.  A verify that stores the state after every token goes step by step.
//
// A CTA of 4 warps holds RPC rows of one (lane, head) in fp32 registers (the lane layout of Split: 8 columns of RL rows a
// lane) and takes the tokens in chunks of up to 16 from shared memory.  Bytes bound it: the state is read once and
// written once.
#pragma once

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
    if (tid <= CT) pw[tid] = tid == 0 ? 1.f : expf((float)tid * ld);
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
    for (int c0 = 0; c0 < n; c0 += CT) {
        const int m = min(CT, n - c0);
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
            if (out >= 0 || c0 + CT < n) {
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

template <int DK, typename InT, typename StT>
cudaError_t launch_linear_dk(const LinearParams& p, cudaStream_t s) {
    using SP = Split<DK>;
    const int CT = p.cu_seqlens != nullptr || p.T > kLinChunk ? kLinChunk : p.T;
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
