// gdn_qk_norm_rope.cu -- RMS norm of every query and key head with the position rotation, in one pass; optionally the
// keys and values quantised into the paged 4-bit cache in the same pass; and the read-back of cached rows.
//
//     y = x / sqrt(mean(x^2) + eps) * w
//     (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * inv_freq[i],  for the R / 2 pairs
//     (i, i + R / 2) or (2 i, 2 i + 1) of the first R dimensions
//
// Each head row is read and written once; at 8192 tokens, HQ 32, HK 8, D 128, bf16, that is 25 us of HBM, and 50 us (3.4 TB/s)
// were measured; in fp32 68 us (50).  Neither the issue slots (60 %) nor DRAM (31 %) are full: after a group's first token each row is
// loaded where it is used, and four CTAs of 64 registers cover part of that.  Few instructions (about 187 a warp for two rows of
// 128) still pay, since they leave more of the time to the loads.  With the store 16381 tokens of that shape take 152 us (66 us of
// HBM with their read-back, which takes 22 us); in fp32 210 us.
// A row belongs to D / 8 lanes of one warp, and a lane holds both numbers of its four pairs (two chunks of 4 dimensions,
// half the rotated part apart), so a rotation exchanges nothing and only the sum of squares is shuffled; the arithmetic is
// two fp32 numbers an instruction.  The angles are those of a token, not of a head: a CTA takes several tokens, forms
// their sines and cosines once in shared memory, and a lane holds its four for all rows of a token.
//
// Angles of far positions: a turn is 2^64, inv_freq becomes a 64-bit fraction of a turn and position * fraction is exact
// modulo 2^64, so the angle is right to 2^-44 turns at position 2^20; its upper 32 bits go through sincospif.
//
// Store: a group of 16 dimensions gets the scale e4m3(max|x| / 6 / k_scale) and codes e2m1(x / scale).  The codes are
// those of the exact value, whatever the order of the sums: the fp32 value carries a bound of its error, and where value
// - bound and value + bound have different codes (or scales) the row is put on a list and formed again at the CTA's end in
// two-float arithmetic (about 2^-44; fp64 instructions are 64 cycles a warp here).  That happens to about one row in
// several hundred.  Values come from storage exactly: their quotients are rounded to odd before the rounding to e4m3 or
// e2m1, which gives what rounding the true quotient gives.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of one CTA
constexpr float kMaxF32 = 3.4028235e38f;

constexpr int kRows = 2;  // of a token that a group of lanes loads together
constexpr int kCtas = 4;  // of an SM: 2 rows and 32 warps an SM beat 4 rows and 16 (8192 tokens 49.5 us against 55.6)

// Four consecutive numbers as two pairs
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    using Raw = uint2;
    __device__ __forceinline__ static Raw load(const __nv_bfloat16* p) {
        Raw r;
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
        return r;
    }
    __device__ __forceinline__ static void unpack(Raw r, F2 (&x)[2]) {
        x[0] = f2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
        x[1] = f2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const F2 (&x)[2]) {
        const float2 a = split(x[0]), b = split(x[1]);
        const __nv_bfloat162 u = __floats2bfloat162_rn(a.x, a.y), v = __floats2bfloat162_rn(b.x, b.y);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
    }
};
template <>
struct Quad<float> {
    using Raw = uint4;
    __device__ __forceinline__ static Raw load(const float* p) { return ld_state16(p); }
    __device__ __forceinline__ static void unpack(Raw r, F2 (&x)[2]) {
        x[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    __device__ __forceinline__ static void store(float* p, const F2 (&x)[2]) {
        const float2 a = split(x[0]), b = split(x[1]);
        *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
    }
};

// ---- two-float arithmetic: h + l, |l| <= ulp(h) / 2 (Dekker, Knuth) --------------------------------------------
struct Df {
    float h, l;
};
__device__ __forceinline__ Df df_norm(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Df df_add(Df a, Df b) {
    const float s = __fadd_rn(a.h, b.h), v = __fadd_rn(s, -a.h);
    const float e = __fadd_rn(__fadd_rn(a.h, -__fadd_rn(s, -v)), __fadd_rn(b.h, -v));
    return df_norm(s, __fadd_rn(e, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Df df_mul(Df a, Df b) {
    const float h = __fmul_rn(a.h, b.h);
    return df_norm(h, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.h, b.h, -h))));
}
__device__ __forceinline__ Df df_neg(Df a) { return {-a.h, -a.l}; }
__device__ constexpr Df df_const(double x) { return {(float)x, (float)(x - (double)(float)x)}; }
// above (1), at (0) or below (-1) the number t
__device__ __forceinline__ int df_side(Df a, float t) {
    const float d = __fadd_rn(__fadd_rn(a.h, -t), a.l);
    return d > 0.f ? 1 : d < 0.f ? -1 : 0;
}

// sine and cosine of a 64-bit fraction of a turn, to about 2^-44: a quarter turn is split off, the Taylor series follows
// (x^17 / 17! < 2^-54 for x <= pi / 4), its first coefficients in two-float arithmetic
__device__ __forceinline__ void df_sincos(uint64_t turn, Df& s, Df& c) {
    const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
    const int64_t r = (int64_t)(turn - ((uint64_t)quarter << 62));
    const float rh = __ll2float_rn(r), rl = __ll2float_rn(r - (int64_t)rh);
    const Df x = df_mul(df_norm(rh * 0x1p-64f, rl * 0x1p-64f), df_const(6.283185307179586476925));
    const Df y = df_mul(x, x);
    float t = 1.f / 1307674368000.f;
    t = __fmaf_rn(-t, y.h, 1.f / 6227020800.f);
    t = __fmaf_rn(-t, y.h, 1.f / 39916800.f);
    Df p = df_add(df_const(1.0 / 362880), df_mul({-t, 0.f}, y));
    p = df_add(df_const(-1.0 / 5040), df_mul(p, y));
    p = df_add(df_const(1.0 / 120), df_mul(p, y));
    p = df_add(df_const(-1.0 / 6), df_mul(p, y));
    const Df sn = df_add(x, df_mul(df_mul(p, y), x));
    t = 1.f / 20922789888000.f;
    t = __fmaf_rn(-t, y.h, 1.f / 87178291200.f);
    t = __fmaf_rn(-t, y.h, 1.f / 479001600.f);
    t = __fmaf_rn(-t, y.h, 1.f / 3628800.f);
    p = df_add(df_const(1.0 / 40320), df_mul({-t, 0.f}, y));
    p = df_add(df_const(-1.0 / 720), df_mul(p, y));
    p = df_add(df_const(1.0 / 24), df_mul(p, y));
    p = df_add(df_const(-0.5), df_mul(p, y));
    const Df cn = df_add({1.f, 0.f}, df_mul(p, y));
    s = quarter & 1 ? cn : sn;
    c = quarter & 1 ? sn : cn;
    if (quarter & 2) s = df_neg(s);
    if ((quarter + 1) & 2) c = df_neg(c);
}

// ---- the 4-bit format -----------------------------------------------------------------------------------------
// a / b rounded to odd: the truncated quotient with its last bit set where something is lost.  Rounding it again to far
// fewer bits gives what rounding the true quotient gives.
__device__ __forceinline__ float div_odd(float a, float b) {
    const float q = __fdiv_rz(a, b);
    return fmaf(q, b, -a) != 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;
}

// 1 / sqrt(x) of a normal number, to 2^-22 (rsqrtf has three instructions more, for subnormal ones); infinity of 0
__device__ __forceinline__ float rsqrt_normal(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The largest magnitude of eight numbers, by their bits: NaN where one is among them, else infinity
__device__ __forceinline__ float largest(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return __uint_as_float(m);
}

// Where a token's row of the cache lies
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

// One frequency as a 64-bit fraction of a turn: inv_freq * 2^64 / (2 pi), by its 24-bit significand and the first 64 bits
// of 4 / (2 pi)
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
    const uint32_t b = __float_as_uint(inv_freq), e = (b >> 23) & 0xffu;
    const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : (uint64_t)(b & 0x7fffffu) << 1;
    const uint64_t f = __umul64hi(m << 40, 0xA2F9836E4E441529ull);
    const int s = 128 - (int)e;  // e 127: one turn is 2 pi
    const uint64_t r = s >= 64 ? 0 : s >= 0 ? f >> s : s > -64 ? f << -s : 0;
    return b >> 31 ? 0 - r : r;
}

// The two chunks of 4 dimensions of lane l of a query or key row, and whether they are rotated: chunks half the rotated
// part apart, or (INTER, and beyond the rotated part) neighbours
template <bool INTER>
struct Chunks {
    int a, b;
    bool rot;
    __device__ __forceinline__ Chunks(int l, int R) {
        const int half = R / 8;
        rot = l < half;
        a = INTER ? 2 * l : rot ? l : R / 4 + 2 * (l - half);
        b = !INTER && rot ? l + half : a + 1;
    }
};

// A row whose squares may leave fp32 is normed after a multiplication by a power of two, 1 / 2^E: 2^E is about the larger of the
// row's largest magnitude `top` (its bits) and sqrt(eps), so that x' = x / 2^E, mean x'^2 and eps' = eps / 2^2E neither overflow nor
// lose a square that counts, and x' / sqrt(mean x'^2 + eps') is the same number.
constexpr float kLeastMean = 0x1p-100f;  // squares below fp32's normal numbers are lost beside it
__device__ __forceinline__ float row_unit(uint32_t top, float eps) {
    const uint32_t of_eps = eps > 0.f ? ((__float_as_uint(eps) >> 23) + 128u) >> 1 : 0u;
    const uint32_t e = min(max(max(top >> 23, of_eps), 1u), 253u);
    return __uint_as_float((254u - e) << 23);
}
// 1 / 2^E of a row of which these lanes hold 8 numbers each
template <int D>
__device__ __forceinline__ float row_unit(const float (&x)[8], float eps, uint32_t gmask) {
    uint32_t top = __float_as_uint(largest(x));
    for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(gmask, top, o));
    return row_unit(top, eps);
}

// One key row in two-float arithmetic, by the D / 8 lanes that hold its dimensions: its codes and scales into the cache.
// `ex`: a place for D / 4 chunks' maxima, of this row's lanes alone.
template <typename T, int D, bool INTER>
__device__ __noinline__ void store_key_exact(const QkNormRopeParams& p, int t, int head, int l, uint32_t gmask, float2* ex) {
    const Chunks<INTER> ch(l, p.R);
    const T* x = (const T*)p.k + (int64_t)t * p.k_stride + (int64_t)head * D;
    const int d[2] = {ch.a * 4, ch.b * 4};
    float v[8];
    for (int j = 0; j < 8; ++j) v[j] = to_f32(x[d[j >> 2] + (j & 3)]);
    const float unit = row_unit<D>(v, p.eps, gmask);
    Df ss{0.f, 0.f};
    for (int j = 0; j < 8; ++j) {
        v[j] *= unit;
        const float q = __fmul_rn(v[j], v[j]);
        ss = df_add(ss, {q, __fmaf_rn(v[j], v[j], -q)});
    }
    for (int o = D / 16; o > 0; o >>= 1) {
        const float h = __shfl_xor_sync(gmask, ss.h, o), lo = __shfl_xor_sync(gmask, ss.l, o);
        ss = df_add(ss, {h, lo});
    }
    const Df mean = df_add({ss.h * (1.f / D), ss.l * (1.f / D)}, {p.eps * unit * unit, 0.f});
    const float r0 = rsqrtf(mean.h);
    const Df one = df_mul(df_mul(mean, {r0, 0.f}), {r0, 0.f});
    const float e = __fadd_rn(__fadd_rn(1.f, -one.h), -one.l);
    const Df rs = df_norm(r0, r0 * e * fmaf(0.375f, e, 0.5f));
    Df z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = df_mul(df_mul({v[j], 0.f}, rs), {p.kw[d[j >> 2] + (j & 3)], 0.f});
    if (ch.rot) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int a = INTER ? 2 * j : j, b = INTER ? 2 * j + 1 : j + 4;
            Df s, c;
            df_sincos((uint64_t)(int64_t)p.positions[t] * turn_fraction(p.inv_freq[4 * l + j]), s, c);
            const Df u = z[a], v = z[b];
            z[a] = df_add(df_mul(u, c), df_neg(df_mul(v, s)));
            z[b] = df_add(df_mul(v, c), df_mul(u, s));
        }
    }
    uint32_t neg = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (z[j].h < 0.f) neg |= 1u << j, z[j] = df_neg(z[j]);
    const int64_t row = row_of(p.kv, slot_of(p.kv, p.slot_map[t]), 0, head);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        Df top{0.f, 0.f};
#pragma unroll
        for (int j = 4 * k; j < 4 * k + 4; ++j)
            if (z[j].h > top.h || (z[j].h == top.h && z[j].l > top.l)) top = z[j];
        ex[k ? ch.b : ch.a] = make_float2(top.h, top.l);
    }
    __syncwarp(gmask);
    const float ks = p.kv.k_scale;  // a power of two
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = k ? ch.b : ch.a;
        Df top{0.f, 0.f};
        for (int i = c & ~3; i < (c & ~3) + 4; ++i) {
            const float2 v = ex[i];
            if (v.x > top.h || (v.x == top.h && v.y > top.l)) top = {v.x, v.y};
        }
        // the scale: the rounded one of top.h, moved where top passes the midpoint above or below it (six times a midpoint
        // has 7 bits: exact)
        uint32_t sb = f32_to_e4m3(top.h / ks * (1.f / 6.f));
        if (sb < 0x7eu) {
            const int above = df_side(top, 3.f * (e4m3_to_f32(sb) + e4m3_to_f32(sb + 1)) * ks);
            if (above > 0 || (above == 0 && (sb & 1))) ++sb;
        }
        if (sb > 0) {
            const int above = df_side(top, 3.f * (e4m3_to_f32(sb) + e4m3_to_f32(sb - 1)) * ks);
            if (above < 0 || (above == 0 && (sb & 1))) --sb;
        }
        const float s = e4m3_to_f32(sb) * ks;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Df v = z[4 * k + j];
            uint32_t code = 0;
            const float border[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
#pragma unroll
            for (int i = 0; i < 7; ++i) code += df_side(v, border[i] * s) >= ((i & 1) ? 0 : 1);  // a tie goes to the even code
            if (s == 0.f) code = 0;
            w |= (code | ((neg >> (4 * k + j)) & 1) << 3) << (4 * j);
        }
        *reinterpret_cast<uint16_t*>(p.kv.codes + row * (D / 2) + c * 2) = (uint16_t)w;
        if ((c & 3) == 0) p.kv.scales[row * (D / 16) + c / 4] = (uint8_t)sb;
    }
    __syncwarp(gmask);
}

template <typename T, int D, bool STORE, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtas)
    gdn_qk_norm_rope_kernel(const __grid_constant__ QkNormRopeParams p, int tokens_per_cta, int rows_per_cta, int side) {
    constexpr int LPR = D / 8, NG = kThreads / LPR;  // lanes of a row, rows side by side
    constexpr int U = kRows;
    extern __shared__ float4 cs4[];                  // cos [tokens][R / 2], sin [tokens][R / 2]
    float* cs = reinterpret_cast<float*>(cs4);
    __shared__ float4 s_w[2][D / 4];  // the weights of queries and keys
    __shared__ float2 s_ex[STORE ? kThreads / 32 : 1][64];
    __shared__ int s_again;  // key rows whose codes fp32 leaves open
    const int tid = threadIdx.x, grp = tid / LPR, l = tid % LPR, H = p.R / 2;
    const int rows = p.HQ + p.HK + (STORE ? p.HK : 0);  // of a token
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, p.N - t0);
    const int r0 = blockIdx.y * rows_per_cta, nr = min(rows_per_cta, rows - r0);
    const uint32_t gmask = LPR == 32 ? ~0u : ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);
    float* sn = cs + tokens_per_cta * H;
    int* again = reinterpret_cast<int*>(sn + tokens_per_cta * H);
    uint32_t bits = 0;
    // this group's rows of each of its tokens: `side` tokens side by side, the rows NG / side apart
    const int step = NG / side, sub = grp / step, mine = grp - sub * step;
    const Chunks<INTER> ch(l, p.R);

    // where a row's two chunks are read (values lie in neighbouring chunks) and written, and the way to the group's next token
    const T* src[U];
    T* dst[U];
    int64_t hop[U], out_hop[U];
    int gap[U];
    bool mine_here[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = mine + u * step + r0;
        const bool q = r < p.HQ, k = r < p.HQ + p.HK;
        const int64_t stride = q ? p.q_stride : k ? p.k_stride : p.v_stride, out_stride = (int64_t)(q ? p.HQ : p.HK) * D;
        T* out = k ? (T*)(q ? p.q_out : p.k_out) : nullptr;
        mine_here[u] = mine + u * step < nr;
        src[u] = (q ? (const T*)p.q + (int64_t)r * D : k ? (const T*)p.k + (int64_t)(r - p.HQ) * D : (const T*)p.v + (int64_t)(r - p.HQ - p.HK) * D) +
                 (t0 + sub) * stride + (k ? ch.a * 4 : l * 8);
        dst[u] = out ? out + (t0 + sub) * out_stride + (int64_t)(q ? r : r - p.HQ) * D + ch.a * 4 : nullptr;
        hop[u] = stride * side;
        out_hop[u] = out ? out_stride * side : 0;
        gap[u] = k ? (ch.b - ch.a) * 4 : 4;
    }
    typename Quad<T>::Raw raw[U][2];
    auto fetch = [&](int i) {  // the group's rows of the CTA's token i
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i < nt && mine_here[u]) {
                raw[u][0] = Quad<T>::load(src[u]);
                raw[u][1] = Quad<T>::load(src[u] + gap[u]);
            }
            src[u] += hop[u];
        }
    };
    fetch(sub);
    // the tokens' angles and the weights, while the first rows are on their way
    if (tid == 0) s_again = 0;
    for (int j = tid; j < D / 2; j += kThreads)
        s_w[j / (D / 4)][j % (D / 4)] = reinterpret_cast<const float4*>(j < D / 4 ? p.qw : p.kw)[j % (D / 4)];
    for (int j = tid; j < nt * H; j += kThreads) {
        const int t = j / H;
        const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + t] * turn_fraction(p.inv_freq[j - t * H]);
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, sn + j, cs + j);
    }
    __syncthreads();

    for (int i = sub; i < nt; i += side) {
        const int t = t0 + i;
        if (i > sub) fetch(i);
        float4 co = make_float4(1.f, 1.f, 1.f, 1.f), si = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ch.rot) {
            co = *reinterpret_cast<const float4*>(cs + i * H + 4 * l);
            si = *reinterpret_cast<const float4*>(sn + i * H + 4 * l);
        }
        const F2 c2[2] = {f2(co.x, co.y), f2(co.z, co.w)}, s2[2] = {f2(si.x, si.y), f2(si.z, si.w)};
        const F2 n2[2] = {f2(-si.x, -si.y), f2(-si.z, -si.w)};
        Slot slot{0, 0, false};
        if (STORE && mine + r0 + (U - 1) * step >= p.HQ) {
            const int32_t s = p.slot_map[t];
            slot = slot_of(p.kv, s);
            if (!slot.ok && s != -1) bits |= GDN_ERRBIT_INDEX;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = mine + u * step + r0;
            if (!mine_here[u]) continue;  // the same for all lanes of a row
            F2 x[2][2];
            Quad<T>::unpack(raw[u][0], x[0]);
            Quad<T>::unpack(raw[u][1], x[1]);
            const bool is_v = STORE && r >= p.HQ + p.HK, is_k = !is_v && r >= p.HQ;
            if (is_v) {
                if constexpr (STORE) {
                    if (!slot.ok) continue;
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = split(x[j >> 1][j & 1]);
                        v[2 * j] = a.x, v[2 * j + 1] = a.y;
                    }
                    float top = largest(v);
                    if (!(top <= kMaxF32)) {
                        bits |= GDN_ERRBIT_NONFINITE;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = v[j] != v[j] ? 0.f : fminf(fmaxf(v[j], -kMaxF32), kMaxF32);
                        top = largest(v);
                    }
                    top = fmaxf(top, __shfl_xor_sync(gmask, top, 1));
                    const uint32_t sb = f32_to_e4m3(div_odd(fminf(top / p.kv.v_scale, kMaxF32), 6.f));
                    const float s = e4m3_to_f32(sb) * p.kv.v_scale, inv = 1.f / s;
                    if (sb == 0x7eu) {  // the largest scale: what passes the codes is cut first, so that no quotient passes the type
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = fminf(fmaxf(v[j], -8.f * s), 8.f * s);
                    }
                    uint32_t w = 0;
                    if (sb) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            float q[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float a = v[j + h], g = a * inv;
                                q[h] = fmaf(fmaf(-g, s, a), inv, g);  // the quotient to half an ulp
                                if constexpr (sizeof(T) == 4) {  // to odd; 16-bit values meet no border but exactly
                                    const float rem = fmaf(-q[h], s, a);
                                    const uint32_t qb = __float_as_uint(q[h]);
                                    if (rem != 0.f) q[h] = __uint_as_float((qb - ((rem < 0.f) != (a < 0.f))) | 1u);
                                }
                            }
                            w |= f32x2_to_e2m1(q[0], q[1]) << (4 * j);
                        }
                    }
                    const int64_t row = row_of(p.kv, slot, 1, r - p.HQ - p.HK);
                    *reinterpret_cast<uint32_t*>(p.kv.codes + row * (D / 2) + l * 4) = w;
                    if ((l & 1) == 0) p.kv.scales[row * (D / 16) + l / 2] = (uint8_t)sb;
                }
                continue;
            }
            auto squares = [&]() {  // of the row
                F2 acc = mul(x[0][0], x[0][0]);
                acc = fma(x[0][1], x[0][1], acc);
                acc = fma(x[1][0], x[1][0], acc);
                acc = fma(x[1][1], x[1][1], acc);
                const float2 two = split(acc);
                float ss = two.x + two.y;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
                return ss;
            };
            float mean = fmaf(squares(), 1.f / D, p.eps);
            if (!(mean >= kLeastMean && mean <= kMaxF32)) {  // the same for all lanes of a row
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = split(x[j >> 1][j & 1]);
                    v[2 * j] = a.x, v[2 * j + 1] = a.y;
                }
                const float unit = row_unit<D>(v, p.eps, gmask);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j >> 1][j & 1] = mul(x[j >> 1][j & 1], f2(unit, unit));
                mean = fmaf(squares(), 1.f / D, p.eps * unit * unit);
            }
            const float rs = rsqrt_normal(mean);
            const F2 rr = f2(rs, rs);
            const float4 wa = s_w[is_k][ch.a], wb = s_w[is_k][ch.b];
            F2 y[2][2], z[2][2];
            y[0][0] = mul(mul(x[0][0], rr), f2(wa.x, wa.y));
            y[0][1] = mul(mul(x[0][1], rr), f2(wa.z, wa.w));
            y[1][0] = mul(mul(x[1][0], rr), f2(wb.x, wb.y));
            y[1][1] = mul(mul(x[1][1], rr), f2(wb.z, wb.w));
#pragma unroll
            for (int j = 0; j < 2; ++j) z[0][j] = y[0][j], z[1][j] = y[1][j];
            if (ch.rot) {
                if constexpr (INTER) {
                    const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = split(y[j >> 1][j & 1]);
                        z[j >> 1][j & 1] = f2(fmaf(a.x, c4[j], -a.y * s4[j]), fmaf(a.y, c4[j], a.x * s4[j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        z[0][j] = fma(y[0][j], c2[j], mul(y[1][j], n2[j]));
                        z[1][j] = fma(y[1][j], c2[j], mul(y[0][j], s2[j]));
                    }
                }
            }
            if (dst[u]) {
                Quad<T>::store(dst[u], z[0]);
                Quad<T>::store(dst[u] + gap[u], z[1]);
                dst[u] += out_hop[u];
            }
            if constexpr (STORE) {
                if (!is_k || !slot.ok) continue;
                const int head = r - p.HQ;
                // e bounds |z - exact|: the sum of squares (4 terms a number in order, then a tree), root and products give y
                // to 2^-20 of itself, the angle is right to 2^-22, and z mixes the two numbers of a pair
                float v[8], e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = split(z[j >> 1][j & 1]), b = split(y[j >> 1][j & 1]);
                    v[2 * j] = a.x, v[2 * j + 1] = a.y;
                    if (INTER) e[j] = fabsf(b.x) + fabsf(b.y);
                }
                if (!INTER) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 a = split(y[0][j]), b = split(y[1][j]);
                        e[2 * j] = fabsf(a.x) + fabsf(b.x);
                        e[2 * j + 1] = fabsf(a.y) + fabsf(b.y);
                    }
                }
                const bool odd = !(largest(v) <= kMaxF32);
                if (odd) {
                    bits |= GDN_ERRBIT_NONFINITE;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] != v[j] ? 0.f : fminf(fmaxf(v[j], -kMaxF32), kMaxF32);
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = e[j] <= kMaxF32 ? e[j] : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) e[j] *= 0x1p-19f;
                auto bound = [&](int j) { return INTER ? e[j >> 1] : e[j & 3]; };
                float lo[2], hi[2];  // between which a chunk's largest lies
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float m = fmaxf(fmaxf(fabsf(v[4 * k]), fabsf(v[4 * k + 1])), fmaxf(fabsf(v[4 * k + 2]), fabsf(v[4 * k + 3])));
                    const float d = INTER ? fmaxf(e[2 * k], e[2 * k + 1]) : fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                    lo[k] = m - d, hi[k] = m + d;
                }
                // the maxima of a group's four chunks, whichever lanes hold them
                float2* ex = s_ex[tid >> 5] + (tid & 31) / LPR * (D / 4);
                ex[ch.a] = make_float2(lo[0], hi[0]);
                ex[ch.b] = make_float2(lo[1], hi[1]);
                __syncwarp(gmask);
                const float inv = 1.f / p.kv.k_scale;  // a power of two: exact
                const int64_t row = row_of(p.kv, slot, 0, head);
                uint32_t diff = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = k ? ch.b : ch.a;
                    const float4 m0 = *reinterpret_cast<const float4*>(ex + (c & ~3)), m1 = *reinterpret_cast<const float4*>(ex + (c & ~3) + 2);
                    const float low = fmaxf(fmaxf(fmaxf(m0.x, m0.z), fmaxf(m1.x, m1.z)), 0.f) * inv * (1.f / 6.f) * (1.f - 0x1p-21f);
                    const float high = fmaxf(fmaxf(m0.y, m0.w), fmaxf(m1.y, m1.w)) * inv * (1.f / 6.f) * (1.f + 0x1p-21f);
                    const uint32_t sb = f32_to_e4m3(low);
                    diff |= sb ^ f32_to_e4m3(high);
                    const float rsc = sb ? inv / e4m3_to_f32(sb) : 0.f;
                    uint32_t w = 0;
#pragma unroll
                    for (int j = 4 * k; j < 4 * k + 4; j += 2) {
                        // the codes of v and of both ends of where the exact value lies.  The bound goes by both numbers of a
                        // pair, so the ends may lie on both sides of 0, and equally far: signs count but for codes of 0
                        const F2 q = mul(f2(v[j], v[j + 1]), f2(rsc, rsc));
                        const float ea = bound(j) * rsc, eb = bound(j + 1) * rsc;
                        const float2 low = split(add(q, f2(-ea, -eb))), high = split(add(q, f2(ea, eb)));
                        const float2 mid = split(q);
                        const uint32_t b0 = f32x2_to_e2m1(low.x, low.y), b1 = f32x2_to_e2m1(high.x, high.y);
                        const uint32_t m0 = b0 & 0x77u;
                        diff |= (b0 ^ b1) & (0x77u | ((m0 + 0x77u) & 0x88u));  // (a magnitude + 7 reaches the sign's bit if it is not 0)
                        w |= (m0 | (mid.x < 0.f ? 8u : 0u) | (mid.y < 0.f ? 0x80u : 0u)) << (4 * (j & 3));
                    }
                    *reinterpret_cast<uint16_t*>(p.kv.codes + row * (D / 2) + c * 2) = (uint16_t)w;
                    if ((c & 3) == 0) p.kv.scales[row * (D / 16) + c / 4] = (uint8_t)sb;
                }
                if (__any_sync(gmask, diff != 0) && !__any_sync(gmask, odd) && l == 0) again[atomicAdd(&s_again, 1)] = i * p.HK + head;
            }
        }
    }
    if constexpr (STORE) {
        __syncthreads();  // the rows' first codes are written
        const int n = s_again;
        for (int a = grp; a < n; a += NG) {
            const int i = again[a] / p.HK;
            store_key_exact<T, D, INTER>(p, t0 + i, again[a] - i * p.HK, l, gmask, s_ex[tid >> 5] + (tid & 31) / LPR * (D / 4));
        }
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);
}

// One group of 16 dimensions a thread: 8 bytes of codes and a scale in, 32 bytes of bf16 out.  A thread keeps its group
// (key or value, head, dimensions) and walks over tokens, kReadTokens at a time for the sake of loads in flight: 16381 tokens
// of HK 8, D 128 take 22 us (67 MB of bf16 and 19 MB of codes; their scattered 64-byte reads and the writes, not the peak, bound it).
constexpr int kReadTokens = 4;

__global__ void __launch_bounds__(kThreads) gdn_kv4_read_kernel(const __grid_constant__ Kv4ReadParams p, int lanes) {
    const int groups = p.kv.D / 16, items = 2 * p.kv.HK * groups, side = kThreads / lanes;
    const int sub = threadIdx.x / lanes, first = threadIdx.x - sub * lanes;
    const int64_t t0 = (int64_t)blockIdx.x * side * kReadTokens + sub;
    uint32_t bits = 0;
    Slot slot[kReadTokens];
#pragma unroll
    for (int i = 0; i < kReadTokens; ++i) {
        const int64_t t = t0 + i * side;
        const int32_t s = t < p.N ? p.slot_map[t] : -1;
        slot[i] = slot_of(p.kv, s);
        if (!slot[i].ok && s != -1) bits |= GDN_ERRBIT_INDEX;
    }
    for (int x = first; x < items; x += lanes) {
        const int g = x & (groups - 1), wh = x / groups, which = wh >= p.kv.HK, head = wh - which * p.kv.HK;
        uint2 codes[kReadTokens];
        uint32_t sb[kReadTokens];
#pragma unroll
        for (int i = 0; i < kReadTokens; ++i) {
            const int64_t at = row_of(p.kv, slot[i], which, head) * groups + g;
            if (slot[i].ok) {
                codes[i] = *reinterpret_cast<const uint2*>(p.kv.codes + at * 8);
                sb[i] = p.kv.scales[at];
            }
        }
#pragma unroll
        for (int i = 0; i < kReadTokens; ++i) {
            if (!slot[i].ok) continue;
            const float sc = e4m3_to_f32(sb[i]) * (which ? p.kv.v_scale : p.kv.k_scale);
            uint32_t out[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t f[4];
                e2m1x8_to_f16(h ? codes[i].y : codes[i].x, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * sc, v.y * sc);
                    out[4 * h + j] = *reinterpret_cast<const uint32_t*>(&b);
                }
            }
            char* dst = (char*)(which ? p.v_out : p.k_out) + (((t0 + i * side) * p.kv.HK + head) * groups + g) * 32;
            st_plain16(dst, make_uint4(out[0], out[1], out[2], out[3]));
            st_plain16(dst + 16, make_uint4(out[4], out[5], out[6], out[7]));
        }
    }
    if (bits && p.err) atomicOr(p.err, (int32_t)bits);
}

int pow2_at_least(int n) {
    int x = 1;
    while (x < n) x *= 2;
    return x;
}

template <typename T, int D, bool STORE, bool INTER>
cudaError_t run(const QkNormRopeParams& p, cudaStream_t s) {
    constexpr int NG = kThreads / (D / 8), U = kRows;
    const int rows = p.HQ + p.HK + (STORE ? p.HK : 0);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // Few tokens: one row a group of lanes, over as many CTAs as that takes, so that no row waits for another.  Many: U
    // rows a group and several tokens a CTA, as far as that leaves every SM four CTAs.
    const bool few = (int64_t)p.N * rows <= (int64_t)sms * 4 * NG;
    const int most = few ? NG : NG * U, rows_cta = rows < most ? rows : most, ny = (rows + rows_cta - 1) / rows_cta;
    const int side = rows_cta <= NG ? NG / pow2_at_least(rows_cta) : 1;
    int64_t tokens = few ? side : (int64_t)p.N * ny / (4 * sms);
    tokens = tokens < side ? side : tokens > kMaxTokens && side <= kMaxTokens ? kMaxTokens : tokens > side && side > kMaxTokens ? side : tokens;
    const dim3 grid((unsigned)((p.N + tokens - 1) / tokens), (unsigned)ny);
    const size_t smem = (size_t)tokens * (p.R * sizeof(float) + (STORE ? p.HK * sizeof(int) : 0));
    gdn_qk_norm_rope_kernel<T, D, STORE, INTER><<<grid, kThreads, smem, s>>>(p, (int)tokens, rows_cta, side);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_d(const QkNormRopeParams& p, cudaStream_t s) {
    if (p.v) return p.interleaved ? run<T, D, true, true>(p, s) : run<T, D, true, false>(p, s);
    return p.interleaved ? run<T, D, false, true>(p, s) : run<T, D, false, false>(p, s);
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
    const int items = 2 * p.kv.HK * (p.kv.D / 16), lanes = items < kThreads ? pow2_at_least(items) : kThreads;
    const int64_t tokens = (int64_t)(kThreads / lanes) * kReadTokens;
    gdn_kv4_read_kernel<<<(unsigned)((p.N + tokens - 1) / tokens), kThreads, 0, s>>>(p, lanes);
    return cudaGetLastError();
}

}  // namespace gdn
