// gdn_qk_norm_rope.cu -- RMS norm of every query and key head with the position rotation, in one pass; optionally the
// keys and values quantised into the paged 4-bit cache in the same pass; and the read-back of cached rows.
//
//     y = x / sqrt(mean(x^2) + eps) * w
//     (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * inv_freq[i],  for the R / 2 pairs
//     (i, i + R / 2) or (2 i, 2 i + 1) of the first R dimensions
//
// HBM bound: each head row is read and written once.  A row belongs to D / 8 lanes of one warp (8 dimensions, one or two
// 16-byte accesses a lane): the sum of squares and the rotation's partners stay in registers and shuffles.  The angles
// are those of a token, not of a head, so a CTA forms a token's R / 2 sines and cosines once in shared memory and its
// rows all use them; per row they would cost more issue slots than the row's memory time.
//
// Angles of far positions: a turn is 2^64, inv_freq becomes a 64-bit fraction of a turn and position * fraction is exact
// modulo 2^64, so the angle is right to 2^-36 turns at position 2^20; its upper 32 bits go through sincospif.
//
// Store: a group of 16 dimensions gets the scale e4m3(max|x| / 6 / k_scale) and codes e2m1(x / scale).  The codes are
// those of the exact value, whatever the order of the sums: the fp32 value carries a bound E of its error, and where
// value - E and value + E have different codes (or scales) the row's lanes form it again in fp64.  That happens to about
// one row in several hundred.  Values come from storage exactly and need no such care: the scale's quotient is rounded to
// odd before its rounding to e4m3, and the codes compare |x| with border * scale, which is exact in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of one CTA
constexpr int kRowsInFlight = 4;  // rows a group of lanes loads before it works on them

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    constexpr int CH = Chunk<T>::CH;
#pragma unroll
    for (int c = 0; c < 8 / CH; ++c) {
        const uint4 r = ld_state16(p + c * CH);
        Chunk<T>::unpack(r, x + c * CH);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    constexpr int CH = Chunk<T>::CH;
#pragma unroll
    for (int c = 0; c < 8 / CH; ++c) st_plain16(p + c * CH, Chunk<T>::pack(x + c * CH));
}

// |x| / 6 or the like, rounded to odd: the truncated quotient with its last bit set where something is lost.  Rounding it
// again to far fewer bits gives what rounding the true quotient gives.
__device__ __forceinline__ float div_odd(float a, float b) {
    const float q = __fdiv_rz(a, b);
    return fmaf(q, b, -a) != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// e2m1 magnitude (0 .. 7) of |x| / s by comparison with the seven midpoints; ties to the even code
template <typename F>
__device__ __forceinline__ uint32_t code_of(F ax, F s) {
    return (uint32_t)(ax > F(0.25) * s) + (uint32_t)(ax >= F(0.75) * s) + (uint32_t)(ax > F(1.25) * s) +
           (uint32_t)(ax >= F(1.75) * s) + (uint32_t)(ax > F(2.5) * s) + (uint32_t)(ax >= F(3.5) * s) +
           (uint32_t)(ax > F(5) * s);
}

// e4m3 byte of a / 6 in fp64, to nearest even, saturating
__device__ __noinline__ uint32_t scale_byte_f64(double a) {
    const double x = a / 6.0;
    if (!(x < 448.0)) return 0x7e;
    int e = x > 0.0 ? ilogb(x) : -7;
    if (e < -6) e = -6;
    const int m = (int)rint(scalbn(x, 3 - e));  // 8 .. 16, or 0 .. 8 for subnormal scales
    return e == -6 ? (uint32_t)m : (uint32_t)(((e + 6) << 3) + m);
}

// Where a token's row of this cache lies; nullptr: the slot is out of range
struct Slot {
    int64_t page;
    int row;
    bool ok;
};
__device__ __forceinline__ Slot slot_of(const Kv4& kv, int32_t slot) {
    const uint32_t page = (uint32_t)slot / (uint32_t)kv.page_size;
    return {(int64_t)page, slot - (int32_t)page * kv.page_size, slot >= 0 && page < (uint32_t)kv.num_pages};
}
__device__ __forceinline__ int64_t row_of(const Kv4& kv, const Slot& s, int which, int head) {
    return ((s.page * 2 + which) * kv.HK + head) * kv.page_size + s.row;
}

// Eight codes in their bytes: this lane's half of a group
__device__ __forceinline__ uint32_t pack_codes(const uint32_t (&c)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= c[i] << (4 * i);
    return w;
}

// Phase of one frequency for one position: the turn's fraction as a 64-bit number
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
    double f = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    return (uint64_t)(f * 18446744073709551616.0);
}

template <typename T, int D, bool STORE>
__global__ void __launch_bounds__(kThreads) gdn_qk_norm_rope_kernel(QkNormRopeParams p, int tokens_per_cta,
                                                                    int rows_per_cta) {
    constexpr int LPR = D / 8, NG = kThreads / LPR;  // lanes of a row, rows side by side
    constexpr int U = kRowsInFlight;
    extern __shared__ float2 cs[];  // [tokens][R / 2] (cos, sin)
    const int tid = threadIdx.x, grp = tid / LPR, l = tid % LPR, H = p.R / 2;
    const int rows = p.HQ + p.HK + (STORE ? p.HK : 0);  // of a token
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, p.N - t0);
    const int r0 = blockIdx.y * rows_per_cta, nr = min(rows_per_cta, rows - r0);
    const int items = nt * nr;
    const uint32_t gmask = LPR == 32 ? ~0u : ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);
    uint32_t bits = 0;

    // the lane's rotation: which half of which pairs its 8 dimensions are
    const int d0 = l * 8;
    const bool rot = d0 < p.R;
    const bool second = !p.interleaved && d0 >= H;  // (of the rotated dimensions)
    const int f0 = p.interleaved ? d0 / 2 : (second ? d0 - H : d0);
    const int partner = (tid & 31) / LPR * LPR + (!rot ? l : second ? l - H / 8 : l + H / 8);

    float x[U][8];
    auto row_ptr = [&](int i, int& t, int& r) {
        t = i / nr;
        r = r0 + i - t * nr;
        t += t0;
        const T* base = r < p.HQ            ? (const T*)p.q + (int64_t)t * p.q_stride + (int64_t)r * D
                        : r < p.HQ + p.HK   ? (const T*)p.k + (int64_t)t * p.k_stride + (int64_t)(r - p.HQ) * D
                                            : (const T*)p.v + (int64_t)t * p.v_stride + (int64_t)(r - p.HQ - p.HK) * D;
        return base + d0;
    };
    for (int i0 = 0; i0 < items; i0 += U * NG) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * NG + grp;
            int t, r;
            if (i < items) load8(row_ptr(i, t, r), x[u]);
        }
        if (i0 == 0) {  // the angles, while the first rows are on their way
            for (int j = tid; j < nt * H; j += kThreads) {
                const int t = j / H;
                const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + t] * turn_fraction(p.inv_freq[j - t * H]);
                float s, c;
                sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
                cs[j] = make_float2(c, s);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * NG + grp;
            if (i >= items) continue;  // the same for all lanes of a row
            int t, r;
            row_ptr(i, t, r);
            const bool is_v = STORE && r >= p.HQ + p.HK, is_k = !is_v && r >= p.HQ;
            Slot slot{0, 0, false};
            if (STORE && r >= p.HQ) {
                const int32_t s = p.slot_map[t];
                slot = slot_of(p.kv, s);
                if (!slot.ok && s != -1) bits |= GDN_ERRBIT_INDEX;
            }
            if (is_v) {
                if constexpr (STORE) {
                    if (!slot.ok) continue;
                    const int head = r - p.HQ - p.HK;
                    float top = 0.f;
                    bool odd = false;
                    float ax[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        odd |= !(fabsf(x[u][j]) <= 3.4028235e38f);
                        ax[j] = x[u][j] == x[u][j] ? fabsf(x[u][j]) : 0.f;
                        top = fmaxf(top, ax[j]);
                    }
                    if (odd) bits |= GDN_ERRBIT_NONFINITE;
                    top = fmaxf(top, __shfl_xor_sync(gmask, top, 1));
                    const uint32_t sb = f32_to_e4m3(div_odd(fminf(top / p.kv.v_scale, 3.4028235e38f), 6.f));
                    const float s = e4m3_to_f32(sb) * p.kv.v_scale;
                    uint32_t c[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        c[j] = (s > 0.f ? code_of(ax[j], s) : 0u) | (x[u][j] < 0.f ? 8u : 0u);
                    const int64_t row = row_of(p.kv, slot, 1, head);
                    *reinterpret_cast<uint32_t*>(p.kv.codes + row * (D / 2) + l * 4) = pack_codes(c);
                    if ((l & 1) == 0) p.kv.scales[row * (D / 16) + l / 2] = (uint8_t)sb;
                }
                continue;
            }
            const float* w = (is_k ? p.kw : p.qw) + d0;
            const float4 wa = *reinterpret_cast<const float4*>(w), wb = *reinterpret_cast<const float4*>(w + 4);
            const float ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[u][j], x[u][j], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
            const float rs = 1.f / sqrtf(ss * (1.f / D) + p.eps);
            float y[8], z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[u][j] * rs * ww[j];
            const float2* ct = cs + (t - t0) * H + f0;
            if (!p.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float other = __shfl_sync(gmask, y[j], partner);
                    z[j] = y[j];
                    if (rot) {
                        const float2 a = ct[j];
                        z[j] = second ? fmaf(y[j], a.x, other * a.y) : fmaf(y[j], a.x, -other * a.y);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    z[j] = y[j];
                    z[j + 1] = y[j + 1];
                    if (rot) {
                        const float2 a = ct[j / 2];
                        z[j] = fmaf(y[j], a.x, -y[j + 1] * a.y);
                        z[j + 1] = fmaf(y[j + 1], a.x, y[j] * a.y);
                    }
                }
            }
            if (!is_k) {
                store8((T*)p.q_out + ((int64_t)t * p.HQ + r) * D + d0, z);
                continue;
            }
            const int head = r - p.HQ;
            if (p.k_out) store8((T*)p.k_out + ((int64_t)t * p.HK + head) * D + d0, z);
            if constexpr (STORE) {
                if (!slot.ok) continue;
                // E bounds |z - exact|: the sum of squares (16 terms a lane in order, then a tree), root, reciprocal and
                // products give y to 2^-20 of itself, the angle is right to 2^-22, and z mixes two of them
                float e[8];
                bool odd = false;
                float top = 0.f, top_e = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float other = p.interleaved ? y[j ^ 1] : __shfl_sync(gmask, y[j], partner);
                    e[j] = 0x1p-19f * (fabsf(y[j]) + (rot ? fabsf(other) : 0.f));
                    odd |= !(fabsf(z[j]) <= 3.4028235e38f);
                    const float az = z[j] == z[j] ? fabsf(z[j]) : 0.f;
                    if (e[j] != e[j]) e[j] = 0.f;
                    top = fmaxf(top, az);
                    top_e = fmaxf(top_e, e[j]);
                }
                if (odd) bits |= GDN_ERRBIT_NONFINITE;
                top = fmaxf(top, __shfl_xor_sync(gmask, top, 1));
                top_e = fmaxf(top_e, __shfl_xor_sync(gmask, top_e, 1));
                const float inv = 1.f / p.kv.k_scale;  // a power of two: exact
                const float lo = fmaxf(top - top_e, 0.f) * inv * (1.f / 6.f), hi = (top + top_e) * inv * (1.f / 6.f);
                uint32_t sb = f32_to_e4m3(lo);
                bool unsure = sb != f32_to_e4m3(hi);
                const float rsc = sb ? inv / e4m3_to_f32(sb) : 0.f;
                uint32_t c[8], diff = 0;
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float a0 = z[j] == z[j] ? fabsf(z[j]) : 0.f, a1 = z[j + 1] == z[j + 1] ? fabsf(z[j + 1]) : 0.f;
                    const uint32_t b0 = f32x2_to_e2m1(fmaxf(a0 - e[j], 0.f) * rsc, fmaxf(a1 - e[j + 1], 0.f) * rsc);
                    const uint32_t b1 = f32x2_to_e2m1((a0 + e[j]) * rsc, (a1 + e[j + 1]) * rsc);
                    diff |= b0 ^ b1;
                    c[j] = b0 & 0xfu;
                    c[j + 1] = b0 >> 4;
                }
                unsure = (unsure || diff != 0) && !odd;
                if (__any_sync(gmask, unsure)) {
                    double sd = 0.0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sd += (double)x[u][j] * (double)x[u][j];
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) sd += __shfl_xor_sync(gmask, sd, o);
                    const double rd = 1.0 / sqrt(sd / D + (double)p.eps);
                    double zd[8], td = 0.0;
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        // this dimension and its partner; selected without indexing registers by j
                        float xj = x[u][0], wj = ww[0], xn = x[u][1], wn = ww[1];
#pragma unroll
                        for (int m = 1; m < 8; ++m) {
                            if (m == j) xj = x[u][m], wj = ww[m];
                            if (m == (j ^ 1)) xn = x[u][m], wn = ww[m];
                        }
                        if (j == 1) xn = x[u][0], wn = ww[0];
                        const double yj = (double)xj * rd * (double)wj;
                        double other = (double)xn * rd * (double)wn;
                        if (!p.interleaved) other = __shfl_sync(gmask, yj, partner);
                        double zj = yj;
                        if (rot) {
                            const uint64_t turn = (uint64_t)(int64_t)p.positions[t] *
                                                  turn_fraction(p.inv_freq[f0 + (p.interleaved ? j / 2 : j)]);
                            double sn, cn;
                            sincospi((double)(int64_t)turn * 0x1p-63, &sn, &cn);
                            const bool hi_half = p.interleaved ? (j & 1) != 0 : second;
                            zj = hi_half ? yj * cn + other * sn : yj * cn - other * sn;
                        }
                        zd[j] = zj;
                        td = fmax(td, fabs(zj));
                    }
                    td = fmax(td, __shfl_xor_sync(gmask, td, 1));
                    sb = scale_byte_f64(td * (double)inv);
                    const double s = (double)e4m3_to_f32(sb) * (double)p.kv.k_scale;
#pragma unroll 1
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t cj = s > 0.0 ? code_of(fabs(zd[j]), s) : 0u;
#pragma unroll
                        for (int m = 0; m < 8; ++m)
                            if (m == j) c[m] = cj;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] |= z[j] < 0.f ? 8u : 0u;
                const int64_t row = row_of(p.kv, slot, 0, head);
                *reinterpret_cast<uint32_t*>(p.kv.codes + row * (D / 2) + l * 4) = pack_codes(c);
                if ((l & 1) == 0) p.kv.scales[row * (D / 16) + l / 2] = (uint8_t)sb;
            }
        }
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);
}

// One group of 16 dimensions a thread: 8 bytes of codes and a scale in, 32 bytes of bf16 out.
__global__ void __launch_bounds__(kThreads) gdn_kv4_read_kernel(Kv4ReadParams p) {
    const int groups = p.kv.D / 16;
    const int64_t total = (int64_t)p.N * 2 * p.kv.HK * groups;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / groups;
        const int g = (int)(i - r * groups);
        const int64_t th = r / p.kv.HK;
        const int head = (int)(r - th * p.kv.HK), which = (int)(th & 1);
        const int64_t t = th >> 1;
        const int32_t s = p.slot_map[t];
        const Slot slot = slot_of(p.kv, s);
        if (!slot.ok) {
            if (s != -1 && p.err) atomicOr(p.err, (int32_t)GDN_ERRBIT_INDEX);
            continue;
        }
        const int64_t row = row_of(p.kv, slot, which, head);
        const uint2 codes = *reinterpret_cast<const uint2*>(p.kv.codes + (row * groups + g) * 8);
        const float sc = e4m3_to_f32(p.kv.scales[row * groups + g]) * (which ? p.kv.v_scale : p.kv.k_scale);
        uint32_t out[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t f[4];
            e2m1x8_to_f16(h ? codes.y : codes.x, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
                const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * sc, v.y * sc);
                out[4 * h + j] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        char* dst = (char*)(which ? p.v_out : p.k_out) + ((t * p.kv.HK + head) * groups + g) * 32;
        st_plain16(dst, make_uint4(out[0], out[1], out[2], out[3]));
        st_plain16(dst + 16, make_uint4(out[4], out[5], out[6], out[7]));
    }
}

template <typename T, int D, bool STORE>
cudaError_t run(const QkNormRopeParams& p, cudaStream_t s) {
    constexpr int NG = kThreads / (D / 8);
    const int rows = p.HQ + p.HK + (STORE ? p.HK : 0);
    // Few tokens: one row a group of lanes, over as many CTAs as that takes, so that no row waits for another.  Many:
    // kRowsInFlight rows a group, which keeps the loads of a row in flight under the work of the one before.
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const bool few = (int64_t)p.N * rows <= (int64_t)sms * 4 * NG;
    const int want = few ? NG : NG * kRowsInFlight;
    int tokens = want / rows;
    tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
    const int rows_cta = rows <= want ? rows : want;
    const dim3 grid((unsigned)((p.N + tokens - 1) / tokens), (unsigned)((rows + rows_cta - 1) / rows_cta));
    gdn_qk_norm_rope_kernel<T, D, STORE>
        <<<grid, kThreads, (size_t)tokens * (p.R / 2) * sizeof(float2), s>>>(p, tokens, rows_cta);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_d(const QkNormRopeParams& p, cudaStream_t s) {
    return p.v ? run<T, D, true>(p, s) : run<T, D, false>(p, s);
}

template <typename T>
cudaError_t run_t(const QkNormRopeParams& p, cudaStream_t s) {
    return p.D == 64 ? run_d<T, 64>(p, s) : p.D == 128 ? run_d<T, 128>(p, s) : run_d<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeParams& p, bool bf16, cudaStream_t s) {
    return bf16 ? run_t<__nv_bfloat16>(p, s) : run_t<float>(p, s);
}

cudaError_t launch_kv4_read(const Kv4ReadParams& p, cudaStream_t s) {
    const int64_t total = (int64_t)p.N * 2 * p.kv.HK * (p.kv.D / 16);
    const int64_t ctas = (total + kThreads - 1) / kThreads;
    gdn_kv4_read_kernel<<<(unsigned)(ctas < 152 * 32 ? ctas : 152 * 32), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
