// The 4-bit K/V cache: store, read back, and attention of new tokens over it.
//
// Format.  Each group of g channels of one position and head keeps
//   z = min x,  s = fp16((max x - min x) / 15),  code = clamp(rint((x - z) / s), 0, 15)
// (x rounded to fp16 first, fp32 IEEE difference and quotient, ties to even)
// and stands for code * s + z.  Layout: kie_kv4.h.
//
// Attention.  With x^ = code * s + z,
//   q . k^_j     = sum_g s_jg (q_g . c_jg) + z_jg sum(q_g)
//   sum_j p_j v^_j = sum_j (p_j s_jg) c_j + sum_j p_j z_jg
// so the codes enter the matrix instructions as they are: a nibble in the low
// mantissa bits of an fp16 is the subnormal code * 2^-24 (2^-20 where it sits 4
// bits higher), an exact operand that costs one AND for two codes.  The powers
// of two move into q for K and to the end for V.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kie_device.cuh"
#include "kie_kv4.h"

using namespace kie;
namespace cg = cooperative_groups;

namespace {

// ---- element types -----------------------------------------------------------------------------
template <int T> struct Elem;
template <> struct Elem<KV4_F16> {
    using type = __half;
    static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};
template <> struct Elem<KV4_BF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<KV4_F32> {
    using type = float;
    static __device__ __forceinline__ float to(float x) { return x; }
    static __device__ __forceinline__ float from(float x) { return x; }
};

// Eight consecutive channels; vec: the address is a multiple of 16 bytes.
template <int T>
__device__ __forceinline__ void load8(const typename Elem<T>::type* p, bool vec, float* f) {
    using E = typename Elem<T>::type;
    if (vec) {
        constexpr int N = 16 / sizeof(E);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + i);
            const E* e = reinterpret_cast<const E*>(&w);
#pragma unroll
            for (int j = 0; j < N; ++j) f[i * N + j] = Elem<T>::to(e[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = Elem<T>::to(p[j]);
    }
}
// N (2 or 4) consecutive channels, vectorised where the address allows.
template <int T, int N>
__device__ __forceinline__ void load_few(const typename Elem<T>::type* p, float* f) {
    using E = typename Elem<T>::type;
    struct alignas(N * sizeof(E)) V { E e[N]; };
    V v;
    if ((reinterpret_cast<uintptr_t>(p) & (sizeof(V) - 1)) == 0) v = *reinterpret_cast<const V*>(p);
    else {
#pragma unroll
        for (int j = 0; j < N; ++j) v.e[j] = p[j];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = Elem<T>::to(v.e[j]);
}
template <int T>
__device__ __forceinline__ void store8(typename Elem<T>::type* p, bool vec, const float* f) {
    using E = typename Elem<T>::type;
    if (vec) {
        constexpr int N = 16 / sizeof(E);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            uint4 w;
            E* e = reinterpret_cast<E*>(&w);
#pragma unroll
            for (int j = 0; j < N; ++j) e[j] = Elem<T>::from(f[i * N + j]);
            reinterpret_cast<uint4*>(p)[i] = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = Elem<T>::from(f[j]);
    }
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Where the scale and the zero of a row's group lie, in fp16 elements of the params
// (rows of a head start at multiples of 64, so a row's place in its block is row % 8).
struct ParAt { size_t s, z; };
__device__ __forceinline__ ParAt par_at(size_t row, int gi, int ng, bool isv) {
    const size_t blk = (row >> 3) * (16 * ng);
    const int r = int(row & 7), e = r >> 2, t = e ? 7 - r : r;
    if (isv) return ParAt{blk + (t * 2 * ng + gi) * 2 + e, blk + (t * 2 * ng + ng + gi) * 2 + e};
    return ParAt{row * (2 * ng) + gi, row * (2 * ng) + ng + gi};
}

// ---- fp16 pairs
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float h_lo(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w))); }
__device__ __forceinline__ float h_hi(uint32_t w) { return __half2float(__ushort_as_half(uint16_t(w >> 16))); }

// ---- store and read back -----------------------------------------------------------------------
// A row (one position of one head, K or V) is D/8 lanes of 8 channels.  A block
// takes RB consecutive rows [token][head] of one request, RPT of them per lane
// group, so that a thread has RPT independent loads in flight.
//
// Both should be bound by memory and are bound by instructions: about 100 for eight
// channels stored and 60 read, so packed arithmetic, values of 16 bits as pairs as far as
// they go, and the general case (infinities, NaN, tiny bf16, quotients next to a half, tiny
// scales) behind a branch.  K and V of 2 x 4,001 tokens of 32 heads of 128 in bf16 (168 MB):
// 62 us stored (82 without those), 38 us read; fp32 (300 MB) 79 and 53 us, 0.57 and 0.84 of
// the copy rate.  One token of 8 requests: 2 us.
constexpr int RPT = 4;
template <int D> __host__ __device__ constexpr int rows_per_block() { return 256 / (D / 8) * RPT; }

struct RowArgs {
    Kv4 c;
    Kv4Strides ks, vs;
    const int32_t *start, *n_tok;
    int32_t n, chunks;       // tokens, blocks per request
    int32_t dt, dh;          // (256 / lanes per row) / heads and its remainder: from a thread's row to its next
};

// A block's request, its tokens and first position; a thread's row: token and head.
struct Where { int b, nt, t, h; int64_t start; };
template <int D>
__device__ __forceinline__ Where where(const RowArgs& A) {
    Where w;
    w.b = int(blockIdx.x) / A.chunks;
    const int r = (int(blockIdx.x) - w.b * A.chunks) * rows_per_block<D>() + threadIdx.x / (D / 8);
    w.t = r / A.c.heads;
    w.h = r - w.t * A.c.heads;
    w.nt = A.n_tok ? min(__ldg(A.n_tok + w.b), A.n) : A.n;
    w.start = __ldg(A.start + w.b);
    return w;
}
// Row of the codes at which the current token is stored; false: it is not.
__device__ __forceinline__ bool stored_at(const RowArgs& A, const Where& w, size_t& row) {
    const int64_t pos = w.start + w.t;
    row = (size_t(w.b) * A.c.heads + w.h) * A.c.ctx_pad + size_t(pos);
    return w.t < w.nt && pos >= 0 && pos < A.c.max_ctx;
}
__device__ __forceinline__ void next_row(const RowArgs& A, Where& w) {
    w.t += A.dt;
    w.h += A.dh;
    if (w.h >= A.c.heads) { w.h -= A.c.heads; ++w.t; }
}

// Eight channels as pairs of 16 bits: bf16 as they are, others in fp16 (not yet saturated).
template <int T>
__device__ __forceinline__ void load_pairs(const typename Elem<T>::type* p, uint32_t* x) {
    if (T != KV4_F32 && aligned16(p)) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else if (T != KV4_F32) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = uint32_t(h[2 * i]) | uint32_t(h[2 * i + 1]) << 16;
    } else {
        float f[8];
        load8<T>(p, aligned16(p), f);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pack_h2(f[2 * i], f[2 * i + 1]);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 pair_f2(uint32_t x) {
    return BF16 ? make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)) : make_float2(h_lo(x), h_hi(x));
}
// Minimum or maximum of pairs; a NaN stays.
template <bool BF16, bool MAX>
__device__ __forceinline__ uint32_t pair_ext(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16 && MAX) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if (MAX) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// d / 15, rounded to nearest even: with y = RN(1/15) and q = RN(d y), within an ulp of the
// quotient, the residual d - 15 q is exact and RN(q + residual y) is RN(d / 15) (P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  d is a difference of fp16 values: no underflow.
__device__ __forceinline__ float div15(float d) {
    constexpr float Y = 1.f / 15.f;
    const float q = d * Y;
    return fmaf(fmaf(-15.f, q, d), Y, q);
}

template <int T, int D, int NG>
__global__ void __launch_bounds__(256) kv4_append_kernel(const RowArgs A, const void* k, const void* v) {
    using E = typename Elem<T>::type;
    constexpr int LPR = D / 8, BLK = D / 32, LPG = LPR / NG;      // lanes per row, blocks, lanes per group
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const bool isv = blockIdx.y != 0;
    const Kv4& c = A.c;
    const Kv4Strides& s = isv ? A.vs : A.ks;
    Where w = where<D>(A);
    size_t row[RPT];
    bool ok[RPT];
    uint32_t x[RPT][4];
    const E* base = static_cast<const E*>(isv ? v : k) + w.b * s.b + l * 8;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        ok[u] = stored_at(A, w, row[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[u][i] = 0u;
        if (ok[u]) load_pairs<T>(base + w.t * s.t + w.h * s.h, x[u]);
        next_row(A, w);
    }
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        if (!__any_sync(0xffffffffu, ok[u])) continue;
        // (minimum, -maximum) of the group in 16 bits each; NaN where there is one
        auto extremes = [&](auto bf16) {
            constexpr bool B = decltype(bf16)::value;
            uint32_t lo2 = x[u][0], hi2 = x[u][0];
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                lo2 = pair_ext<B, false>(lo2, x[u][i]);
                hi2 = pair_ext<B, true>(hi2, x[u][i]);
            }
            hi2 ^= 0x80008000u;
            uint32_t r = pair_ext<B, false>(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
            for (int o = 1; o < LPG; o <<= 1) r = pair_ext<B, false>(r, __shfl_xor_sync(0xffffffffu, r, o));
            return r;
        };
        // A bf16 of 2^-17 or more is an fp16 as it is (7 bits of fraction, the last at 2^-24)
        constexpr bool B16 = T == KV4_BF16;
        float2 f[4];                 // the values in fp32
        uint32_t mm = extremes(std::integral_constant<bool, B16>());
        float2 ext = pair_f2<B16>(mm);
        bool plain = fmaxf(fabsf(ext.x), fabsf(ext.y)) <= 65504.f && ext.x + ext.y <= 65504.f;     // false for a NaN in x or y
        if (B16) {
            uint32_t a = x[u][0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < 4; ++i) a = __vminu2(a, x[u][i] & 0x7FFF7FFFu);
            plain = plain && min(a & 0xFFFFu, a >> 16) >= 0x3700u;                                 // 2^-17
        }
        if (__any_sync(0xffffffffu, !plain)) {                   // to fp16, saturated to +-65504, NaN as 0
            const __half2 top = __half2half2(__ushort_as_half(0x7BFF)), bottom = __half2half2(__ushort_as_half(0xFBFF));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = pair_f2<B16>(x[u][i]);
                const __half2 h = __floats2half2_rn(y.x, y.y);
                uint32_t bits = *reinterpret_cast<const uint32_t*>(&h) & __heq2_mask(h, h);
                const __half2 r = __hmax2(__hmin2(*reinterpret_cast<__half2*>(&bits), top), bottom);
                x[u][i] = *reinterpret_cast<const uint32_t*>(&r);
                f[i] = pair_f2<false>(x[u][i]);
            }
            mm = extremes(std::false_type());
            ext = pair_f2<false>(mm);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = pair_f2<B16>(x[u][i]);
        }
        const float lo = ext.x, span = -ext.y - lo;
        const __half sh = __float2half_rn(div15(span));
        const float sf = __half2float(sh);
        float rcp;                   // 0 for a constant group: all codes 0
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rcp) : "f"(sf));
        if (!(sf > 0.f)) rcp = 0.f;
        // code = rint((x - z) / s): by the reciprocal, which is within 2^-18 of the quotient, so
        // only a value that close to a half needs the division itself.  Adding 1.5 * 2^23 rounds
        // to even.  A normal s is within 2^-11 of its quotient and the codes end at 15; a
        // subnormal one's are limited.
        constexpr float MAGIC = 12582912.f;
        const float2 magic = make_float2(MAGIC, MAGIC), rcp2 = make_float2(rcp, rcp), neg = make_float2(-lo, -lo);
        float2 d[4], n[4];           // n: codes, negated
        float far = 0.f;             // largest distance from a code
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = __fadd2_rn(f[i], neg);
            n[i] = __ffma2_rn(__ffma2_rn(d[i], rcp2, magic), make_float2(-1.f, -1.f), magic);
            const float2 e = __ffma2_rn(d[i], rcp2, n[i]);
            far = fmaxf(far, fmaxf(fabsf(e.x), fabsf(e.y)));
        }
        if (far > 0.5f - 1.f / 65536.f || (sf < 6.103515625e-5f && sf > 0.f)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                n[i].x = -fminf(rintf(__fdiv_rn(d[i].x, sf)), 15.f);
                n[i].y = -fminf(rintf(__fdiv_rn(d[i].y, sf)), 15.f);
            }
        }
        // sum of code_i 16^i, in two halves of 16 bits
        const float2 b256 = make_float2(256.f, 256.f);
        const float2 w0 = __ffma2_rn(n[1], b256, n[0]), w1 = __ffma2_rn(n[3], b256, n[2]);
        const uint32_t word = __byte_perm(__float_as_uint(fmaf(w0.y, -16.f, MAGIC - w0.x)),
                                          __float_as_uint(fmaf(w1.y, -16.f, MAGIC - w1.x)), 0x5410);
        if (!isv) {
            if (ok[u]) reinterpret_cast<uint32_t*>(c.kc)[row[u] * LPR + (l & 3) * BLK + (l >> 2)] = word;
        } else {
            // lane l stores word l = units (g, 2wi) and (g, 2wi + 1): see kie_kv4.h
            const int g = l / (D / 64), wi = l % (D / 64);
            const int src = (lane - l) + 8 * wi + (g >> 1);
            const uint32_t v0 = __shfl_sync(0xffffffffu, word, src), v1 = __shfl_sync(0xffffffffu, word, src + 4);
            if (ok[u]) reinterpret_cast<uint32_t*>(c.vc)[row[u] * LPR + l] = __byte_perm(v0, v1, (g & 1) ? 0x7632 : 0x5410);
        }
        if (ok[u] && l % LPG == 0) {
            const ParAt at = par_at(row[u], l / LPG, NG, isv);
            uint16_t* pp = isv ? c.vp : c.kp;
            pp[at.s] = __half_as_ushort(sh);
            pp[at.z] = __half_as_ushort(__float2half_rn(lo));
        }
    }
}

template <int T, int D, int NG>
__global__ void __launch_bounds__(256) kv4_read_kernel(const RowArgs A, void* k, void* v) {
    using E = typename Elem<T>::type;
    constexpr int LPR = D / 8, BLK = D / 32, LPG = LPR / NG;
    const int l = threadIdx.x % LPR;
    const bool isv = blockIdx.y != 0;
    const Kv4& c = A.c;
    const Kv4Strides& st = isv ? A.vs : A.ks;
    Where w = where<D>(A);
    bool ok[RPT];
    uint32_t word[RPT], sz[RPT];
    const Where w0 = w;
    const uint32_t* kc = reinterpret_cast<const uint32_t*>(c.kc) + (l & 3) * BLK + (l >> 2);
    const uint16_t* vc = reinterpret_cast<const uint16_t*>(c.vc) + (2 * (l & 3)) * BLK + (l >> 2);
    const uint16_t* pp = isv ? c.vp : c.kp;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        size_t row;
        ok[u] = stored_at(A, w, row);
        next_row(A, w);
        if (!ok[u]) continue;
        if (!isv) word[u] = __ldg(kc + row * LPR);
        else word[u] = uint32_t(__ldg(vc + row * (D / 4))) | uint32_t(__ldg(vc + row * (D / 4) + BLK)) << 16;
        const ParAt at = par_at(row, l / LPG, NG, isv);
        sz[u] = uint32_t(__ldg(pp + at.s)) | uint32_t(__ldg(pp + at.z)) << 16;
    }
    w = w0;
    E* base = static_cast<E*>(isv ? v : k) + w.b * st.b + l * 8;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        if (ok[u]) {
            const float2 p = h2_to_f2(sz[u]), ps = make_float2(p.x, p.x), pz = make_float2(p.y, p.y);
            const uint32_t even = word[u] & 0x0F0F0F0Fu, odd = (word[u] >> 4) & 0x0F0F0F0Fu;
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {      // 2^23 + code comes of the bits
                const float2 big = make_float2(__uint_as_float(__byte_perm(even, 0x4B000000u, 0x7540 + i)),
                                               __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7540 + i)));
                const float2 y = __ffma2_rn(__fadd2_rn(big, make_float2(-8388608.f, -8388608.f)), ps, pz);
                f[2 * i] = y.x;
                f[2 * i + 1] = y.y;
            }
            E* q = base + w.t * st.t + w.h * st.h;
            if (T == KV4_F16) {
                uint4 o;
                __half2* h = reinterpret_cast<__half2*>(&o);
                const __half2 top = __half2half2(__ushort_as_half(0x7BFF)), bottom = __half2half2(__ushort_as_half(0xFBFF));
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = __hmax2(__hmin2(__floats2half2_rn(f[2 * i], f[2 * i + 1]), top), bottom);
                if (aligned16(q)) *reinterpret_cast<uint4*>(q) = o;
                else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i] = reinterpret_cast<const E*>(&o)[i];
                }
            } else {
                store8<T>(q, aligned16(q), f);
            }
        }
        next_row(A, w);
    }
}

// ---- attention ---------------------------------------------------------------------------------
// An item is a pair (request, tile of RT query rows) and a K/V head; its work is
// the tiles of TP positions that some row of it sees.  Two forms:
//   cluster  an item belongs to a cluster of CTAs that split its tiles and join
//            their (m, l, o) through distributed shared memory: one launch;
//   stream   the tiles of all items form one list that is cut into equal ranges,
//            one per CTA, whatever the requests' lengths; a CTA leaves a partial
//            (m, l, o) of each item that it does not hold whole, and a second
//            kernel joins the partials.
// Long contexts are bound by memory: 8 requests x 16 heads over 32,768 keys, bf16 (671 MB)
// 111 us, 0.89 of the copy rate; there the integer pipe, which takes the codes apart, is
// half busy.  Short ones by latency: an item's chain (lengths, queries, first tiles, the
// join) is 4 us, a second launch 5 more.  16 heads over 32,768 keys in fp16 24 us (floor 11), 8
// ragged requests of up to 8,191 keys 19 (6), 16 heads over 2,300 in fp32 10.3 (0.9).
constexpr int TP = 32;        // positions per tile = one warp's step
// Six warps with two tiles each and two CTAs per SM: 60 to 120 KB in flight per SM.  8 x 2 tiles
// took 10.4 us for 9.9 (16 heads over 2,300 keys, fp32) and 24.9 for 23.5 (32,768 keys, fp16);
// 8 x 3 14.4 and 30.9 (one CTA per SM), 4 x 4 9.6 and 25.4; three CTAs of 6 warps spill: 10.7
// and 32.0.
constexpr int NW = 6;         // warps per CTA, each with its own tiles and copies in flight
constexpr int STG = 2;        // tiles in flight per warp
constexpr int MAXS = 8;       // CTAs per cluster

// Both products run transposed, the cache as the 16-row operand and the query
// rows as the 8 columns: S^T = K q^T, o^T = V^T p^T.  A warp's accumulators then
// hold 8 rows and nothing else, and each unpacked code is used once.
// HL8: 8 query rows, the operands q and p as fp16 hi + lo (22 bits and more: fp32
// and fp16 tensors).  S8, S16: 8 or 16 rows, one fp16 each (bf16 tensors: 11 bits
// are 8 times finer than their rounding).
enum Mode { HL8 = 0, S8 = 1, S16 = 2 };
__host__ __device__ constexpr int rows_of(int mode) { return mode == S16 ? 16 : 8; }
// CTAs per SM: 128 registers a thread do for all but 16 rows of 128 channels.
__host__ __device__ constexpr int ctas_per_sm(int mode, int dim) { return mode == S16 && dim == 128 ? 1 : 2; }

struct AttnArgs {
    Kv4Attn a;
    int32_t per;             // query heads per K/V head
    int32_t nrt;             // row tiles per request
    int32_t nctas;           // stream: CTAs of the main kernel; cluster: CTAs per item
};

// The keys that the rows [r0, r0 + rt) of request b see, as positions [lo, hi).
__device__ __forceinline__ void pair_keys(const AttnArgs& A, int b, int r0, int rt, int& lo, int& hi, int& len, int& n) {
    len = min(max(__ldg(A.a.kv_len + b), 0), A.a.c.max_ctx);
    n = A.a.n_tok ? min(max(__ldg(A.a.n_tok + b), 0), A.a.n_q) : A.a.n_q;
    const int rows = n * A.per;
    lo = hi = 0;
    if (r0 >= rows) return;
    hi = len;
    if (A.a.causal) {
        const int t0 = r0 / A.per, t1 = (min(r0 + rt, rows) - 1) / A.per;
        hi = max(0, len - n + t1 + 1);
        if (A.a.window > 0) lo = max(0, len - n + t0 + 1 - A.a.window);
        if (lo >= hi) lo = hi = 0;
    }
}
__device__ __forceinline__ int key_tiles(int lo, int hi) { return hi > lo ? (hi + TP - 1) / TP - lo / TP : 0; }
__device__ __forceinline__ int pair_tiles(const AttnArgs& A, int p, int rt) {
    int lo, hi, len, n;
    pair_keys(A, p / A.nrt, (p % A.nrt) * rt, rt, lo, hi, len, n);
    return key_tiles(lo, hi);
}

// First tile of CTA i's range, of T tiles over n CTAs (fewer than n where T is: no range is empty).
__device__ __forceinline__ int list_ctas(int64_t T, int n) { return int(min(T, int64_t(n))); }
__device__ __forceinline__ int64_t range_begin(int64_t T, int i, int n) { return i >= n ? T : T * i / n; }

// One warp: total tiles, and the pair that holds the first tile `at` of CTA i (with the pair's first tile).
__device__ __forceinline__ int64_t scan_pairs(const AttnArgs& A, int rt, int i, int& pair, int64_t& first, int64_t& at) {
    const int lane = threadIdx.x & 31, np = A.a.c.batch * A.nrt;
    const int own0 = lane < np ? pair_tiles(A, lane, rt) : 0;     // the first 32 pairs, kept
    int64_t T = own0;
    for (int p0 = 32; p0 < np; p0 += 32) T += p0 + lane < np ? pair_tiles(A, p0 + lane, rt) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    T *= A.a.c.heads;
    at = range_begin(T, i, list_ctas(T, A.nctas));
    pair = np;
    first = T;
    int64_t run = 0;
    for (int p0 = 0; p0 < np; p0 += 32) {
        const int64_t own = int64_t(p0 == 0 ? own0 : p0 + lane < np ? pair_tiles(A, p0 + lane, rt) : 0) * A.a.c.heads;
        int64_t inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, run + inc > at);
        if (hit) {
            const int w = __ffs(hit) - 1;
            pair = p0 + w;
            first = __shfl_sync(0xffffffffu, run + inc - own, w);
            break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
    }
    return T;
}

__device__ __forceinline__ void mma16816(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// The same onto a zero accumulator.
__device__ __forceinline__ void mma16816_0(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Maximum that keeps a NaN, so that a NaN score reaches its row's output.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127
// Four code pairs of a word whose halves hold two elements' nibbles: element
// values code * 2^-24 * {1, 16, 1, 16}.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t* r) {
    r[0] = w & 0x000F000Fu;
    r[1] = w & 0x00F000F0u;
    r[2] = (w >> 8) & 0x000F000Fu;
    r[3] = (w >> 8) & 0x00F000F0u;
}
// The same as normal numbers (code - SUB) * {1, 16, 1, 16}: 1024 + code comes of the bits as well,
// and the subtraction is exact.
template <int SUB>
__device__ __forceinline__ void unpack4_normal(uint32_t w, uint32_t* r) {
    constexpr uint32_t BIG = 0x64006400u;                              // 1024
    r[0] = (w & 0x000F000Fu) | BIG;
    r[1] = (w & 0x00F000F0u) | BIG;
    r[2] = ((w >> 8) & 0x000F000Fu) | BIG;
    r[3] = ((w >> 8) & 0x00F000F0u) | BIG;
    constexpr uint32_t OFF = 0xE400E400u + SUB * 0x00010001u, OFF16 = 0xE400E400u + 16 * SUB * 0x00010001u;   // -(1024 + SUB), -(1024 + 16 SUB)
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("add.rn.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(i & 1 ? OFF16 : OFF));
}
template <bool NORMAL, int SUB>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t* r) {
    if (NORMAL) unpack4_normal<SUB>(w, r);
    else unpack4(w, r);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// Transpose of the warp's 8 x 8 fp16 matrix (lane 4r + c holds row r, columns 2c and 2c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int D, int NG>
struct Tile {
    static constexpr int CODES = TP * D / 2, PAR = TP * 4 * NG, BYTES = 2 * (CODES + PAR);
};

// NG consecutive words (one load).
template <int NG> struct Words { uint32_t w[NG]; };
template <int NG>
__device__ __forceinline__ Words<NG> load_words(const uint8_t* p) {
    Words<NG> r;
    if constexpr (NG == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
    return r;
}

// What the warps of a CTA share, after their rings.
template <int D, int NG, int MODE>
struct AttnShared {
    static constexpr int RT = rows_of(MODE), BLK = D / 32;
    uint4 q[BLK][MODE == S8 ? 1 : 2][32];   // operands of q: [block][rows + 8 (S16) or rest (HL8)][lane], two mmas each
    float qsum[BLK][RT];          // row sums of q per block
    int32_t qexp[RT];             // exponents of the rows' largest elements
    float recv[RT * D];           // cluster: [CTA][RT * D / CTAs] sums of this CTA's stretch of the elements
    float2 recv_ml[MAXS][RT];     // and every CTA's (m, l) of the rows
    int64_t plan[4];
};

template <int D, int NG, int MODE, int T, bool CLUSTER>
__global__ void __launch_bounds__(NW * 32, ctas_per_sm(MODE, D)) kv4_attention_kernel(const AttnArgs A) {
    using E = typename Elem<T>::type;
    using TL = Tile<D, NG>;
    constexpr int RT = rows_of(MODE), BLK = D / 32, BPG = BLK / NG;   // 32-channel blocks, per group
    constexpr int NT = RT / 8;                                        // tiles of 8 query rows
    // fp32 tensors.  The matrix unit aligns what it adds by the operands' exponents and cuts it 24
    // bits below the largest; a subnormal counts there as 2^-14, so of products of codes as
    // subnormals 14 to 18 bits are left, enough for 16-bit results only: here codes become
    // normal numbers (one addition more).  Then K and V are taken as s (code - 8) + (z + 8 s),
    // since over a long context sum p s code and sum p z are some 50 times what they add up to;
    // and only the sums of 16 positions are the matrix unit's, rounded sums of those the rest.
    // Off, of standard normal keys and values: 6e-5 of the result at 2,300 without the three,
    // 8e-6 without the second, 2e-7 with both; at 65,536 8e-6 without the third, 3e-7 with it: no
    // more than plain fp32 sums.  They took 2,300 keys from 9.9 to 10.6 us (10.0 since a warp's
    // sums have memory of their own).  The low parts of q have sums of their own, else each of
    // their products is cut at the large ones' sum: 1.7e-6 -> 8e-7 off with keys whose channels
    // differ tenfold, for 0.3 us.
    constexpr bool FINE = T == KV4_F32;
    extern __shared__ __align__(128) uint8_t smem[];
    AttnShared<D, NG, MODE>& S = *reinterpret_cast<AttnShared<D, NG, MODE>*>(smem);
    uint8_t* const pool = smem + (sizeof(S) + 127) / 128 * 128;       // rings; then every warp's sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = pool + warp * (STG * TL::BYTES);
    const uint32_t ring_u = smem_u32(ring);
    const Kv4& c = A.a.c;

    int pair = 0, head = 0;
    const int rank = CLUSTER ? int(blockIdx.x) % A.nctas : 0;
    if (CLUSTER) {
        if (A.nctas > 1) cg::this_cluster().barrier_arrive();   // waited for before the first remote write
        const int item = int(blockIdx.x) / A.nctas;
        pair = item / c.heads;
        head = item % c.heads;
    } else {
        if (warp == 0) {
            int64_t f, x;
            int p;
            const int64_t total = scan_pairs(A, RT, blockIdx.x, p, f, x);
            if (lane == 0) {
                S.plan[0] = x;
                S.plan[1] = range_begin(total, blockIdx.x + 1, list_ctas(total, A.nctas));
                S.plan[2] = p;
                S.plan[3] = f;
            }
        }
        __syncthreads();
        // let the joining kernel's blocks come up: they wait for this grid's end
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    // stream: the list's state (next tile, end, pair, the pair's first tile) stays in S.plan
    while (true) {
        if (!CLUSTER) {
            if (S.plan[0] >= S.plan[1]) break;
            pair = int(S.plan[2]);
        }
        const int b = pair / A.nrt, r0 = (pair % A.nrt) * RT;
        // ---- the query rows: warp w holds row w (and w + NW), a lane EPL channels; loaded first,
        // their latency passes with that of the lengths
        constexpr int EPL = D / 32, RPW = (RT + NW - 1) / NW;
        float qx[RPW][EPL];
        auto load_q = [&]() {
#pragma unroll
            for (int k = 0; k < RPW; ++k) {
                const int r = r0 + warp + k * NW;
#pragma unroll
                for (int j = 0; j < EPL; ++j) qx[k][j] = 0.f;
                if (warp + k * NW < RT && r < A.a.n_q * A.per) {
                    const int tok = r / A.per, hq = head * A.per + r - tok * A.per;
                    load_few<T, EPL>(static_cast<const E*>(A.a.q) + b * A.a.qs.b + tok * A.a.qs.t + hq * A.a.qs.h + lane * EPL, qx[k]);
                }
            }
        };
        if (CLUSTER) load_q();
        int lo, hi, len, n_new;
        pair_keys(A, b, r0, RT, lo, hi, len, n_new);
        const int nt = key_tiles(lo, hi);
        int tile0, ntile;
        if (CLUSTER) {
            if (r0 >= n_new * A.per) {                // no such rows: the whole cluster leaves
                if (A.nctas > 1) cg::this_cluster().barrier_wait();
                return;
            }
            tile0 = int(int64_t(nt) * rank / A.nctas);
            ntile = int(int64_t(nt) * (rank + 1) / A.nctas) - tile0;
        } else {
            const int64_t at = S.plan[0], first = S.plan[3], pt = int64_t(nt) * c.heads;
            if (at >= first + pt) {
                __syncthreads();
                if (threadIdx.x == 0) { S.plan[2] = pair + 1; S.plan[3] = first + pt; }
                __syncthreads();
                continue;
            }
            head = int((at - first) / nt);
            tile0 = int((at - first) - int64_t(head) * nt);
            ntile = int(min(int64_t(nt - tile0), S.plan[1] - at));
            load_q();
        }
        const int base = lo / TP * TP + tile0 * TP;           // first position of this segment
        const size_t row0 = (size_t(b) * c.heads + head) * c.ctx_pad;
        // this lane's 16-byte pieces of the tiles; V's land with halves of rows 2, 3, 6 and 7
        // of each block swapped (D = 128), which spreads their reads over the banks
        const uint8_t* const kcs = c.kc + (row0 + base) * (D / 2) + lane * 16;
        const uint8_t* const vcs = c.vc + (row0 + base) * (D / 2) + lane * 16;
        const uint8_t* const kps = reinterpret_cast<const uint8_t*>(c.kp) + (row0 + base) * (4 * NG) + lane * 16;
        const uint8_t* const vps = reinterpret_cast<const uint8_t*>(c.vp) + (row0 + base) * (4 * NG) + lane * 16;
        const uint32_t kdst = ring_u + lane * 16;
        const uint32_t vdst = ring_u + TL::CODES + (D == 128 ? (lane * 16) ^ ((lane & 8) << 2) : lane * 16);
        auto copy_tile = [&](int i, int st) {      // tile i of the segment into ring stage st
            const size_t off = size_t(i) * TL::CODES;
            const uint32_t d = st * TL::BYTES;
#pragma unroll
            for (int j = 0; j < TL::CODES / 512; ++j) {
                copy16(kdst + d + j * 512, kcs + off + j * 512);
                copy16(vdst + d + j * 512, vcs + off + j * 512);
            }
            if (lane < TL::PAR / 16) {
                copy16(kdst + d + 2 * TL::CODES, kps + size_t(i) * TL::PAR);
                copy16(kdst + d + 2 * TL::CODES + TL::PAR, vps + size_t(i) * TL::PAR);
            }
        };
#pragma unroll
        for (int s = 0; s < STG - 1; ++s) {
            if (warp + s * NW < ntile) copy_tile(warp + s * NW, s);
            cp_async_commit();
        }

        // ---- the query rows as operands
#pragma unroll
        for (int k = 0; k < RPW; ++k) {
            const int row = warp + k * NW;
            if (row < RT) {                           // uniform over the warp
                const bool have = r0 + row < n_new * A.per;
                float mx = 0.f;
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    if (!have) qx[k][j] = 0.f;
                    mx = fmaxf(mx, fabsf(qx[k][j]));
                }
                // exact power of two that brings the row's largest element to [2^11, 2^12)
                const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
                const int e = min(max(int(mb >> 23) - 127, -100), 114);
                const float up = copysignf(pow2i(11 - e), A.a.scale);
                // channel 32 i + 8 tt + j: half j >> 2 of slot j & 3 of block i, lane (row, tt); the odd
                // slots' codes are 16 times as large
                const int d0 = lane * EPL, i = d0 >> 5, tt = (d0 >> 3) & 3;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    const float y = qx[k][j] * up, h = __half2float(__float2half_rn(y));
                    const int s8 = (d0 + j) & 7;
                    const float f = (s8 & 1) ? 1.f / 16.f : 1.f;
                    sum += y;
                    reinterpret_cast<__half*>(&S.q[i][row >> 3][4 * (row & 7) + tt])[2 * (s8 & 3) + (s8 >> 2)] = __float2half_rn(h * f);
                    if (MODE == HL8)
                        reinterpret_cast<__half*>(&S.q[i][MODE == HL8 ? 1 : 0][4 * row + tt])[2 * (s8 & 3) + (s8 >> 2)] = __float2half_rn((y - h) * f);
                }
#pragma unroll
                for (int d = 1; d < 32 / EPL; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);   // over the block's lanes
                if ((d0 & 31) == 0) S.qsum[i][row] = sum * (1.f / 256.f);
                if (lane == 0) S.qexp[row] = e;
            }
        }
        __syncthreads();
        // the zeros' operand of row g: k = 2t, 2t+1 are a pair of groups (NG == 1: scale and
        // zero), the sums' fp16 for t < 2, their rest after
        uint32_t qz[NT];
        float2 cq[NT];                 // rows 2t, 2t+1: from the mma's units to log2 units of the softmax
        int last[NT][2], firstk[NT][2];     // keys they see: firstk .. last
        int all_lo = 0, all_hi = 1 << 30;   // positions that every row of the tile sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float sum[NG];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                sum[gi] = 0.f;
#pragma unroll
                for (int j = 0; j < BPG; ++j) sum[gi] += S.qsum[gi * BPG + j][g + nt * 8];
            }
            float s0 = 0.f, s1 = 0.f;
            if (NG == 4) { s0 = (t & 1) ? sum[2 % NG] : sum[0]; s1 = (t & 1) ? sum[3 % NG] : sum[1 % NG]; }
            if (NG == 2 && (t & 1) == 0) { s0 = sum[0]; s1 = sum[1 % NG]; }
            if (NG == 1 && (t & 1) == 0) s1 = sum[0];
            const float h0 = __half2float(__float2half_rn(s0)), h1 = __half2float(__float2half_rn(s1));
            qz[nt] = t < 2 ? pack_h2(h0, h1) : pack_h2(s0 - h0, s1 - h1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 2 * t + e + nt * 8, r = r0 + row;
                const bool have = r < n_new * A.per;
                last[nt][e] = !have ? -1 : A.a.causal ? len - n_new + r / A.per : len - 1;
                firstk[nt][e] = A.a.window > 0 && A.a.causal ? last[nt][e] - A.a.window + 1 : 0;
                if (have) { all_lo = max(all_lo, firstk[nt][e]); all_hi = min(all_hi, last[nt][e]); }
                // above 0: it keeps -inf
                (e ? cq[nt].y : cq[nt].x) = fmaxf(fabsf(A.a.scale) * 1.4426950408889634f * pow2i(S.qexp[row] - 11 + (FINE ? 0 : 24)), 1.2e-38f);
            }
        }
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);
        // this lane's places in a block of 8 positions: K row of operand row g, V rows t and 7 - t
        const int krow = g & 1 ? 7 - (g >> 1) : g >> 1;
        const int koff = krow * (D / 2) + t * (D / 8);
        const int v0off = t * (D / 2) + (D == 128 ? (g * 8) ^ ((t & 2) << 4) : g * 4);
        const int v1off = (7 - t) * (D / 2) + (D == 128 ? (g * 8) ^ (((7 - t) & 2) << 4) : g * 4);

        float o[NT][BLK][2][4];        // o^T: [block][nibbles 2jj (c0, c1) and 2jj + 1 (c2, c3)], columns 2t, 2t + 1
        float zl[NT][4];               // row g < NG: sum of p z of group g, row NG: sum of p
        float2 m[NT];
        int ev = 1;                    // biased fp16 exponent of the largest V scale so far
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                zl[nt][k] = 0.f;
#pragma unroll
                for (int i = 0; i < BLK; ++i) o[nt][i][0][k] = o[nt][i][1][k] = 0.f;
            }
        }

        // Every warp's (o, z and l, m) so far: [warp][RT][D], [warp][RT][8], [warp][RT].  What the
        // matrix unit cuts off its sums is cut to one side, so they move there after FLUSH tiles
        // (fp32 tensors' are rounded sums already).  262,144 normal keys and values, without
        // and with it: fp16 3.5e-3 / 5e-4 of the result off, bf16 3.3e-3 / 1.9e-3.  8 x 16
        // heads over 32,768, bf16: 110 us without, 111 at 32, 113 at 16; fp16 16 heads 23.4, 24.2 at 8.
        constexpr int FLUSH = MODE == HL8 ? 8 : 32;
        float* const mo = reinterpret_cast<float*>(pool + NW * STG * TL::BYTES);
        float* const mz = mo + NW * RT * D;
        float* const mm = mz + NW * RT * 8;
        bool flushed = false;
        auto flush = [&]() {
            const float back = pow2i(ev - 14) * (FINE ? 1.f : 16777216.f);   // undo fv and the codes' 2^-24
            float f[NT][2];
#pragma unroll
            for (int nt8 = 0; nt8 < NT; ++nt8)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float old = flushed ? mm[warp * RT + nt8 * 8 + 2 * t + e] : -INFINITY;
                    f[nt8][e] = old == -INFINITY ? 0.f : ex2(old - (e ? m[nt8].y : m[nt8].x));
                }
            __syncwarp();
#pragma unroll
            for (int nt8 = 0; nt8 < NT; ++nt8)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = warp * RT + nt8 * 8 + 2 * t + e;
#pragma unroll
                    for (int i = 0; i < BLK; ++i) {
                        float4* const at = reinterpret_cast<float4*>(mo + size_t(row) * D + i * 32 + g * 4);
                        float4 v = make_float4(o[nt8][i][0][e] * back, o[nt8][i][0][2 + e] * (back * 0.0625f),
                                               o[nt8][i][1][e] * back, o[nt8][i][1][2 + e] * (back * 0.0625f));
                        if (flushed) {
                            const float4 w = *at;
                            v.x = fmaf(f[nt8][e], w.x, v.x);
                            v.y = fmaf(f[nt8][e], w.y, v.y);
                            v.z = fmaf(f[nt8][e], w.z, v.z);
                            v.w = fmaf(f[nt8][e], w.w, v.w);
                        }
                        *at = v;
                    }
                    const float z = FINE ? zl[nt8][e] + zl[nt8][2 + e] : zl[nt8][e];
                    mz[row * 8 + g] = flushed ? fmaf(f[nt8][e], mz[row * 8 + g], z) : z;
                    if (g == 0) mm[row] = e ? m[nt8].y : m[nt8].x;
                }
#pragma unroll
            for (int nt8 = 0; nt8 < NT; ++nt8)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    zl[nt8][k] = 0.f;
#pragma unroll
                    for (int i = 0; i < BLK; ++i) o[nt8][i][0][k] = o[nt8][i][1][k] = 0.f;
                }
            flushed = true;
            __syncwarp();
        };

        int st = 0, kept = 0;
        for (int i = warp; i < ntile; i += NW) {
            {
                const int nx = i + (STG - 1) * NW;
                int ns = st + STG - 1;
                if (ns >= STG) ns -= STG;
                __syncwarp();          // every lane is done with the stage that this overwrites
                if (nx < ntile) copy_tile(nx, ns);
                cp_async_commit();
            }
            if (!FINE && kept++ == FLUSH) {
                flush();
                kept = 1;
            }
            cp_async_wait_group<STG - 1>();
            __syncwarp();
            const uint8_t* kc = ring + st * TL::BYTES;
            const uint8_t* vc = kc + TL::CODES;
            const uint8_t* kp = vc + TL::CODES;
            const uint8_t* vp = kp + TL::PAR;
            if (++st == STG) st = 0;
            const int p0 = base + i * TP;
            if (p0 + TP > len) {       // parameters that nothing was stored to: zeros for V (K's scores are masked)
                if (p0 + lane >= len) {
                    uint16_t* v = reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(vp));
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        const ParAt at = par_at(lane, gi, NG, true);
                        v[at.s] = 0;
                        v[at.z] = 0;
                    }
                }
                __syncwarp();
            }
            // ---- scores of 2 x 16 positions, in units of cq: x[half][block][tile] = rows (2t, 2t+1) of position krow
            float2 x[2][2][NT];
            Words<BLK> w[4];
            Words<NG> par[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                w[n] = load_words<BLK>(kc + n * 4 * D + koff);
                par[n] = load_words<NG>(kp + (n * 8 + krow) * 4 * NG);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                // zeros of this lane's pair of groups (NG == 1: beside the scale, whose factor is 0)
                auto zero = [&](const Words<NG>& q) { return NG == 4 ? ((t & 1) ? q.w[3 % NG] : q.w[2 % NG]) : q.w[NG - 1]; };
                uint4 az = make_uint4(zero(par[2 * hh]), zero(par[2 * hh + 1]), 0u, 0u);
                if (FINE) {                // z + 8 s in two parts, the second at k = 8 ..
                    auto centre = [&](const Words<NG>& q, uint32_t& z, uint32_t& low) {
                        const uint32_t s = NG == 4 ? ((t & 1) ? q.w[1 % NG] : q.w[0]) : NG == 2 ? q.w[0] : q.w[0] << 16;
                        const float a = NG == 1 ? 0.f : fmaf(8.f, h_lo(s), h_lo(z)), b = fmaf(8.f, h_hi(s), h_hi(z));
                        z = pack_h2(a, b);
                        low = pack_h2(a - h_lo(z), b - h_hi(z));
                    };
                    centre(par[2 * hh], az.x, az.z);
                    centre(par[2 * hh + 1], az.y, az.w);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float z[4];
                    mma16816_0(z, az, qz[nt], FINE ? qz[nt] : 0u);
                    constexpr float UNIT = FINE ? 256.f : 1.f / 65536.f;
                    x[hh][0][nt] = make_float2(z[0] * UNIT, z[1] * UNIT);
                    x[hh][1][nt] = make_float2(z[2] * UNIT, z[3] * UNIT);
                }
            }
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                float acc[2][NT][4], low[2][4];      // FINE: products of q's low parts in sums of their own
#pragma unroll
                for (int j = 0; j < BPG; ++j) {
                    const int i2 = gi * BPG + j;
                    uint4 qf[NT], ql;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) qf[nt] = S.q[i2][nt][lane];
                    if (MODE == HL8) ql = S.q[i2][MODE == HL8 ? 1 : 0][lane];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t ra[4], rb[4];
                        unpack<FINE, 8>(w[2 * hh].w[i2], ra);
                        unpack<FINE, 8>(w[2 * hh + 1].w[i2], rb);
                        const uint4 a0 = make_uint4(ra[0], rb[0], ra[1], rb[1]), a1 = make_uint4(ra[2], rb[2], ra[3], rb[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (j == 0) mma16816_0(acc[hh][nt], a0, qf[nt].x, qf[nt].y);
                            else mma16816(acc[hh][nt], a0, qf[nt].x, qf[nt].y);
                            mma16816(acc[hh][nt], a1, qf[nt].z, qf[nt].w);
                        }
                        if (FINE) {
                            if (j == 0) mma16816_0(low[hh], a0, ql.x, ql.y);
                            else mma16816(low[hh], a0, ql.x, ql.y);
                            mma16816(low[hh], a1, ql.z, ql.w);
                        } else if (MODE == HL8) {
                            mma16816(acc[hh][0], a0, ql.x, ql.y);
                            mma16816(acc[hh][0], a1, ql.z, ql.w);
                        }
                    }
                }
                if (FINE) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[hh][0][k] += low[hh][k];
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t sw = par[2 * hh + k].w[gi >> 1];
                        const float s = gi & 1 ? h_hi(sw) : h_lo(sw);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            x[hh][k][nt] = __ffma2_rn(make_float2(acc[hh][nt][2 * k], acc[hh][nt][2 * k + 1]), make_float2(s, s), x[hh][k][nt]);
                    }
            }
            if (p0 < all_lo || p0 + TP - 1 > all_hi) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int p = p0 + hh * 16 + k * 8 + krow;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (p < firstk[nt][0] || p > last[nt][0]) x[hh][k][nt].x = -INFINITY;
                            if (p < firstk[nt][1] || p > last[nt][1]) x[hh][k][nt].y = -INFINITY;
                        }
                    }
            }
            // ---- running maximum, and the largest V scale of the tile
            float2 corr[NT], mref[NT];
            bool grew = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float2 mx = x[0][0][nt];
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    mx.x = max_nan(mx.x, x[k >> 1][k & 1][nt].x);
                    mx.y = max_nan(mx.y, x[k >> 1][k & 1][nt].y);
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    mx.x = max_nan(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, d));
                    mx.y = max_nan(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, d));
                }
                const float2 mn = make_float2(max_nan(m[nt].x, mx.x * cq[nt].x), max_nan(m[nt].y, mx.y * cq[nt].y));
                grew |= mn.x > m[nt].x || mn.y > m[nt].y;
                // p <= 2^15: fp16's range, used whole (fp32 tensors: by a product, as exponents near
                // 15 are rounded to 2^-21)
                constexpr float UP = FINE ? 0.f : 15.f;
                mref[nt] = make_float2((mn.x == -INFINITY ? 0.f : mn.x) - UP, (mn.y == -INFINITY ? 0.f : mn.y) - UP);
                corr[nt] = make_float2(ex2(m[nt].x - UP - mref[nt].x), ex2(m[nt].y - UP - mref[nt].y));
                m[nt] = mn;
            }
            uint32_t sb;
            {
                const Words<NG> v = load_words<NG>(vp + (lane & 15) * 8 * NG);   // pair lane % 16 of the tile
                uint32_t a = v.w[0];
#pragma unroll
                for (int gi = 1; gi < NG; ++gi) a = __vmaxu2(a, v.w[gi]);
                sb = max(a & 0xFFFFu, a >> 16);
            }
            const int en = max(ev, int(__reduce_max_sync(0xffffffffu, sb) >> 10));
            if (__any_sync(0xffffffffu, grew) || en > ev) {
                const float fe = pow2i(ev - en);
                ev = en;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    zl[nt][0] *= corr[nt].x;
                    zl[nt][1] *= corr[nt].y;
                    if (FINE) { zl[nt][2] *= corr[nt].x; zl[nt][3] *= corr[nt].y; }
                    const float cx = corr[nt].x * fe, cy = corr[nt].y * fe;
#pragma unroll
                    for (int i2 = 0; i2 < BLK; ++i2)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            o[nt][i2][j][0] *= cx; o[nt][i2][j][1] *= cy;
                            o[nt][i2][j][2] *= cx; o[nt][i2][j][3] *= cy;
                        }
                }
            }
            const float fv = pow2i(14 - ev);    // 2^-(E+1), E = ev - 15: p * s * fv < 2^15
            const uint32_t fv2 = pack_h2(fv, fv);
            // ---- o^T += v^T p^T, 16 positions at a time
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const uint8_t* va = vc + hh * 8 * D, *vb = va + 4 * D;          // codes and params of the two blocks
                const uint8_t* pa = vp + hh * 64 * NG + t * 8 * NG, *pb = pa + 32 * NG;
                // p as the operand: row g, positions (t, 7 - t) of the two blocks
                uint32_t ph[NT][2], pl[2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 y = x[hh][k][nt];
                        constexpr float UP = FINE ? 32768.f : 1.f;
                        const float px = ex2(fmaf(y.x, cq[nt].x, -mref[nt].x)) * UP, py = ex2(fmaf(y.y, cq[nt].y, -mref[nt].y)) * UP;
                        const uint32_t h = pack_h2(px, py);
                        ph[nt][k] = transpose8(h);
                        if (MODE == HL8) pl[k] = transpose8(pack_h2(px - h_lo(h), py - h_hi(h)));
                    }
                {   // zeros and the row sum: rows 0..NG-1 are the groups' zeros, row NG is 1
                    uint32_t z0 = g == NG ? 0x3C003C00u : 0u, z1 = z0, l0 = 0u, l1 = 0u;
                    if (g < NG) {
                        z0 = *reinterpret_cast<const uint32_t*>(pa + 4 * NG + 4 * g);
                        z1 = *reinterpret_cast<const uint32_t*>(pb + 4 * NG + 4 * g);
                        if (FINE) {        // z + 8 s in two fp16 parts, the second in rows 8 ..
                            auto centre = [](uint32_t s, uint32_t& z, uint32_t& l) {
                                const float a = fmaf(8.f, h_lo(s), h_lo(z)), b = fmaf(8.f, h_hi(s), h_hi(z));
                                z = pack_h2(a, b);
                                l = pack_h2(a - h_lo(z), b - h_hi(z));
                            };
                            centre(*reinterpret_cast<const uint32_t*>(pa + 4 * g), z0, l0);
                            centre(*reinterpret_cast<const uint32_t*>(pb + 4 * g), z1, l1);
                        }
                    }
                    const uint4 az = make_uint4(z0, l0, z1, l1);
                    if (FINE) {
                        float f[4], low[4];
                        mma16816_0(f, az, ph[0][0], ph[0][1]);
                        mma16816_0(low, az, pl[0], pl[1]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) zl[0][k] += f[k] + low[k];
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(zl[nt], az, ph[nt][0], ph[nt][1]);
                        if (MODE == HL8) mma16816(zl[0], az, pl[0], pl[1]);
                    }
                }
                const Words<NG> sa = load_words<NG>(pa), sb2 = load_words<NG>(pb);
                Words<D / 64> vw[4];
                vw[0] = load_words<D / 64>(va + v0off);
                vw[1] = load_words<D / 64>(va + v1off);
                vw[2] = load_words<D / 64>(vb + v0off);
                vw[3] = load_words<D / 64>(vb + v1off);
                uint32_t b[NT][2], bl[2];
#pragma unroll
                for (int i2 = 0; i2 < BLK; ++i2) {
                    if (i2 % BPG == 0) {     // p * s of the group, below 2^15
                        const uint32_t s[2] = {hmul2(sa.w[i2 / BPG], fv2), hmul2(sb2.w[i2 / BPG], fv2)};   // exact, below 1
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) b[nt][k] = hmul2(ph[nt][k], s[k]);
                            // the product's rest is exact in fp16; the low part's product joins it
                            if (MODE == HL8) bl[k] = hfma2(pl[k], s[k], hfma2(ph[0][k], s[k], b[0][k] ^ 0x80008000u));
                        }
                    }
                    const int wi = i2 >> 1;
                    const uint32_t sel = (i2 & 1) ? 0x7632u : 0x5410u;
                    uint32_t u0[4], u1[4];
                    unpack<FINE, 8>(__byte_perm(vw[0].w[wi], vw[1].w[wi], sel), u0);
                    unpack<FINE, 8>(__byte_perm(vw[2].w[wi], vw[3].w[wi], sel), u1);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 a = make_uint4(u0[2 * j], u0[2 * j + 1], u1[2 * j], u1[2 * j + 1]);
                        if (FINE) {
                            float f[4];
                            mma16816_0(f, a, b[0][0], b[0][1]);
                            mma16816(f, a, bl[0], bl[1]);
                            float* const oo = o[0][i2][j];
#pragma unroll
                            for (int k = 0; k < 4; ++k) oo[k] += f[k];
                        } else {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i2][j], a, b[nt][0], b[nt][1]);
                            if (MODE == HL8) mma16816(o[0][i2][j], a, bl[0], bl[1]);
                        }
                    }
                }
            }
        }
        // ---- merge the warps
        cp_async_wait_group<0>();
        flush();
        __syncthreads();
        const bool whole = CLUSTER ? A.nctas == 1 : ntile == nt;
        float* part = A.a.ws + (size_t(pair) * c.heads + head + blockIdx.x) * (RT * (D + 2));
        // four channels of a row, by 1 / ls
        auto store = [&](int r, int d, float4 v, float ls) {
            const int row = r0 + r;
            if (row < n_new * A.per) {
                const int tok = row / A.per;
                E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + tok * A.a.os.t + (head * A.per + row - tok * A.per) * A.a.os.h + d;
                const float f[4] = {v.x, v.y, v.z, v.w};
                struct alignas(4 * sizeof(E)) V { E e[4]; } w;
#pragma unroll
                for (int j = 0; j < 4; ++j) w.e[j] = Elem<T>::from(ls == 0.f ? 0.f : f[j] / ls);
                if ((reinterpret_cast<uintptr_t>(op) & (sizeof(V) - 1)) == 0) *reinterpret_cast<V*>(op) = w;
                else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) op[j] = w.e[j];
                }
            }
        };
        cg::cluster_group cl = cg::this_cluster();
        if (CLUSTER && A.nctas > 1) cl.barrier_wait();        // every CTA of the cluster runs
        const int per = CLUSTER ? RT * D / A.nctas : 1;       // elements that a CTA of the cluster joins
        for (int i = threadIdx.x * 4; i < RT * D; i += NW * 128) {
            const int r = i / D, d = i % D;
            float M = -INFINITY, mw[NW];
#pragma unroll
            for (int w = 0; w < NW; ++w) { mw[w] = mm[w * RT + r]; M = max_nan(M, mw[w]); }
            float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
            float ls = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = mw[w] == -INFINITY ? 0.f : ex2(mw[w] - M);
                const float4 v = *reinterpret_cast<const float4*>(mo + (w * RT + r) * D + d);
                const float z = mz[(w * RT + r) * 8 + d / (D / NG)];
                ls = fmaf(f, mz[(w * RT + r) * 8 + NG], ls);
                os.x = fmaf(f, v.x + z, os.x);
                os.y = fmaf(f, v.y + z, os.y);
                os.z = fmaf(f, v.z + z, os.z);
                os.w = fmaf(f, v.w + z, os.w);
            }
            if (whole) {
                store(r, d, os, ls);
            } else if (CLUSTER) {      // to the CTA that joins these elements
                *reinterpret_cast<float4*>(cl.map_shared_rank(S.recv, i / per) + rank * per + i % per) = os;
                if (d < 4 * A.nctas) cl.map_shared_rank(&S, d / 4)->recv_ml[rank][r] = make_float2(M, ls);
            } else {
                *reinterpret_cast<float2*>(part + i) = make_float2(os.x, os.y);
                *reinterpret_cast<float2*>(part + i + 2) = make_float2(os.z, os.w);
                if (d == 0) *reinterpret_cast<float2*>(part + RT * D + 2 * r) = make_float2(M, ls);
            }
        }
        if (CLUSTER && A.nctas > 1) {
            cl.sync();
            for (int j = threadIdx.x * 4; j < per; j += NW * 128) {
                const int i = rank * per + j, r = i / D;
                float M = -INFINITY, mk[MAXS], lk[MAXS];
#pragma unroll
                for (int k = 0; k < MAXS; ++k) {
                    const float2 ml = k < A.nctas ? S.recv_ml[k][r] : make_float2(-INFINITY, 0.f);
                    mk[k] = ml.x;
                    lk[k] = ml.y;
                    M = max_nan(M, mk[k]);
                }
                float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
                float ls = 0.f;
#pragma unroll
                for (int k = 0; k < MAXS; ++k) {
                    if (k < A.nctas) {
                        const float f = mk[k] == -INFINITY ? 0.f : ex2(mk[k] - M);
                        const float4 v = *reinterpret_cast<const float4*>(S.recv + k * per + j);
                        ls = fmaf(f, lk[k], ls);
                        os.x = fmaf(f, v.x, os.x);
                        os.y = fmaf(f, v.y, os.y);
                        os.z = fmaf(f, v.z, os.z);
                        os.w = fmaf(f, v.w, os.w);
                    }
                }
                store(r, i % D, os, ls);
            }
        }
        if (CLUSTER) break;
        if (threadIdx.x == 0) S.plan[0] += ntile;
        __syncthreads();               // the sums have been read
    }
}

// Join the partials of every item that more than one CTA worked on; items
// without a key get zeros.  One block per (pair, K/V head) and 256 elements.
template <int D, int RT, int T>
__global__ void __launch_bounds__(256) kv4_join_kernel(const AttnArgs A) {
    using E = typename Elem<T>::type;
    __shared__ int64_t s_at[2];
    constexpr int PER = RT * D / 256;
    const int item = blockIdx.x / PER, pair = item / A.a.c.heads, head = item % A.a.c.heads;
    if (threadIdx.x < 32) {
        // tiles of the pairs before this one, and of all
        const int np = A.a.c.batch * A.nrt;
        int64_t before = 0, T_ = 0;
        for (int p = threadIdx.x; p < np; p += 32) {
            const int k = pair_tiles(A, p, RT);
            T_ += k;
            before += p < pair ? k : 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            T_ += __shfl_xor_sync(0xffffffffu, T_, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        if (threadIdx.x == 0) { s_at[0] = before * A.a.c.heads; s_at[1] = T_ * A.a.c.heads; }
    }
    __syncthreads();
    const int64_t total = s_at[1];
    int lo, hi, len, n_new;
    const int b = pair / A.nrt, r0 = (pair % A.nrt) * RT;
    pair_keys(A, b, r0, RT, lo, hi, len, n_new);
    const int i = int(blockIdx.x % PER) * 256 + threadIdx.x, r = i / D, d = i % D, row = r0 + r;
    const int nt = key_tiles(lo, hi);
    int c0 = 0, c1 = 0;                 // CTAs c0 .. c1 hold tiles of this item
    if (nt > 0) {
        const int64_t t0 = s_at[0] + int64_t(head) * nt, t1 = t0 + nt;
        const int n = list_ctas(total, A.nctas);
        // CTA of tile x: the largest i with total * i / n <= x
        auto owner = [&](int64_t x) {
            int k = int((x * n) / total);
            while (k + 1 < n && range_begin(total, k + 1, n) <= x) ++k;
            while (k > 0 && range_begin(total, k, n) > x) --k;
            return k;
        };
        c0 = owner(t0);
        c1 = owner(t1 - 1);
    }
    // every block waits for the main kernel, also one with nothing to join: what
    // follows in the stream waits for this kernel alone
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= n_new * A.per || (nt > 0 && c0 == c1)) return;   // one CTA held it whole and wrote the result
    const float* part = A.a.ws + (size_t(pair) * A.a.c.heads + head) * (RT * (D + 2));
    float M = -INFINITY, ls = 0.f, os = 0.f;
    constexpr int U = 8;                // partials in flight
    for (int k0 = c0; nt > 0 && k0 <= c1; k0 += U) {
        float mk[U], lk[U], ok[U], mn = M;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float* pk = part + size_t(min(k0 + k, c1)) * (RT * (D + 2));
            mk[k] = __ldcg(pk + RT * D + 2 * r);
            lk[k] = __ldcg(pk + RT * D + 2 * r + 1);
            ok[k] = __ldcg(pk + i);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (k0 + k > c1) mk[k] = -INFINITY;
            mn = max_nan(mn, mk[k]);
        }
        const float f = M == -INFINITY ? 0.f : ex2(M - mn);
        ls *= f;
        os *= f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float fk = mk[k] == -INFINITY ? 0.f : ex2(mk[k] - mn);
            ls = fmaf(lk[k], fk, ls);
            os = fmaf(ok[k], fk, os);
        }
        M = mn;
    }
    const int tok = row / A.per;
    E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + tok * A.a.os.t + (head * A.per + row - tok * A.per) * A.a.os.h;
    op[d] = Elem<T>::from(ls == 0.f ? 0.f : os / ls);
}

int mode_of(int type, int rows) { return type != KV4_BF16 ? HL8 : rows <= 8 ? S8 : S16; }

// Shared-memory opt-in of a kernel, once per device.
template <typename K>
cudaError_t opt_in(K* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (r == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
    return r;
}

// How an attention runs, by what the host knows: the mode, the row tiles and the form.
struct Plan {
    int mode, per, nrt, nctas;
    int64_t items;
    int S;                   // CTAs per item of the cluster form; 0: stream form
    double us;               // modelled time
};
Plan plan_of(const Kv4Attn& a, int sms) {
    Plan p;
    p.per = a.heads / a.c.heads;
    const int64_t rows = int64_t(a.n_q) * p.per;
    p.mode = mode_of(a.type, rows > 8 ? 16 : 8);
    const int rt = rows_of(p.mode);
    p.nrt = int((rows + rt - 1) / rt);
    p.nctas = sms * ctas_per_sm(p.mode, a.c.dim);
    p.items = int64_t(a.c.batch) * p.nrt * a.c.heads;
    int64_t keys = a.c.max_ctx;                          // the most that an item can have
    if (a.window > 0) keys = std::min<int64_t>(keys, int64_t(a.window) + (rt + p.per - 1) / p.per + TP);
    const int64_t tiles = (keys + TP - 1) / TP;
    // Cluster form: waves of items, each a start and an end and its warps' tiles in turn.
    // Stream form: evenly cut tiles, but a second launch and an end for each item that a CTA
    // works on; for few items only.  Measured at 128 channels (cluster / stream, us): 16 heads
    // over 2,300 keys fp32 10.4 / 11.9; 8 x 8 over 8,191 bf16 20 / 24; 8 over 32,768 fp32 39 /
    // 20, 8 x 16 125 / 108; 4 rows of 4 heads to each of 8 x 8 over 8,191 60 / 39.  More items
    // than CTAs: 1,024 over 2,300 101 / 124, 512 over 32,768 729 / 683.
    p.S = 1;
    // clusters of 8 fill 120 of the 152 SMs with one CTA each, 288 of 304 with two
    const int64_t room = p.nctas == sms ? p.nctas * 3 / 4 : p.nctas * 15 / 16;
    while (p.S < MAXS && p.S * NW < tiles && p.items * p.S * 2 <= room) p.S *= 2;
    const bool wide = p.mode == S16;
    const double tile = (wide ? 1.25 : p.mode == HL8 ? 1.9 : 1.4) * a.c.dim / 128;
    const double cluster = double((p.items * p.S + p.nctas - 1) / p.nctas) * ((wide ? 6.0 : 5.0) + tile * double((tiles + p.S * NW - 1) / (p.S * NW)));
    const double stream = 6.0 + (wide ? 11.0 : 5.0) * (1.0 + double(p.items) / p.nctas) + tile * double(p.items) * double(tiles) / (p.nctas * NW);
    p.us = cluster;
    if (p.items <= p.nctas && stream < cluster) {
        p.S = 0;
        p.us = stream;
    }
    return p;
}

// Whether the kernel of 256-row tiles (kie_kv4_chunk.cu) takes the call: where its modelled
// time is the smaller.  Measured at 128 channels, group 64 (rows: this / that): 8 x 16 heads
// over 4,096 keys 16: 42 / 52 us, 64: 136 / 54; 8 heads over 32,768 keys 32: 38 / 39, 128:
// 105 / 45; 8 heads over 4,096 keys 64: 21 / 23, 512: 71 / 46.
bool many_tokens(const Kv4Attn& a, int sms) {
    return a.type == KV4_BF16 && int64_t(a.n_q) * (a.heads / a.c.heads) > 16 && plan_of(a, sms).us > kie_kv4_chunk_us(&a, sms);
}

template <int D, int NG, int MODE, int T>
cudaError_t launch_attention(AttnArgs A, const Plan& p, cudaStream_t st) {
    constexpr int RT = rows_of(MODE);
    constexpr int ring = NW * STG * Tile<D, NG>::BYTES, merge = NW * RT * (D + 9) * 4;
    constexpr int smem = (int(sizeof(AttnShared<D, NG, MODE>)) + 127) / 128 * 128 + ring + merge;
    static std::atomic<uint64_t> done{0}, done_c{0};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (p.S) {
        A.nctas = p.S;
        cudaError_t r = opt_in(kv4_attention_kernel<D, NG, MODE, T, true>, smem, done_c);
        if (r != cudaSuccess) return r;
        cfg.gridDim = dim3(unsigned(p.items * p.S));
        cfg.blockDim = dim3(NW * 32);
        cfg.dynamicSmemBytes = smem;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = p.S;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<D, NG, MODE, T, true>, A);
    }
    A.nctas = p.nctas;
    cudaError_t r = opt_in(kv4_attention_kernel<D, NG, MODE, T, false>, smem, done);
    if (r != cudaSuccess) return r;
    kv4_attention_kernel<D, NG, MODE, T, false><<<A.nctas, NW * 32, smem, st>>>(A);
    r = cudaGetLastError();
    if (r != cudaSuccess) return r;
    cfg.gridDim = dim3(unsigned(p.items * (RT * D / 256)));
    cfg.blockDim = dim3(256);
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, RT, T>, A);
}

template <int D, int NG>
cudaError_t launch_attention_t(const AttnArgs& A, const Plan& p, cudaStream_t st) {
    if (A.a.type == KV4_F16) return launch_attention<D, NG, HL8, KV4_F16>(A, p, st);
    if (A.a.type == KV4_F32) return launch_attention<D, NG, HL8, KV4_F32>(A, p, st);
    return p.mode == S8 ? launch_attention<D, NG, S8, KV4_BF16>(A, p, st) : launch_attention<D, NG, S16, KV4_BF16>(A, p, st);
}

template <int D>
RowArgs row_args(const Kv4& c, const Kv4Strides& ks, const Kv4Strides& vs, int n, const int32_t* start,
                 const int32_t* n_tok) {
    constexpr int step = 256 / (D / 8);
    return RowArgs{c, ks, vs, start, n_tok, n, int((int64_t(n) * c.heads + rows_per_block<D>() - 1) / rows_per_block<D>()),
                   step / c.heads, step % c.heads};
}
template <int D, int NG, int T>
cudaError_t rows_t(const RowArgs& A, bool read, void* k, void* v, cudaStream_t st) {
    const dim3 grid(unsigned(A.chunks) * A.c.batch, 2);
    if (read) kv4_read_kernel<T, D, NG><<<grid, 256, 0, st>>>(A, k, v);
    else kv4_append_kernel<T, D, NG><<<grid, 256, 0, st>>>(A, k, v);
    return cudaGetLastError();
}
template <int D, int NG>
cudaError_t rows_ng(const RowArgs& A, int type, bool read, void* k, void* v, cudaStream_t st) {
    if (type == KV4_F16) return rows_t<D, NG, KV4_F16>(A, read, k, v, st);
    if (type == KV4_BF16) return rows_t<D, NG, KV4_BF16>(A, read, k, v, st);
    return rows_t<D, NG, KV4_F32>(A, read, k, v, st);
}
cudaError_t rows(const Kv4& c, void* k, void* v, const Kv4Strides& ks, const Kv4Strides& vs, int type, bool read, int n,
                 const int32_t* start, const int32_t* n_tok, cudaStream_t st) {
    const int ng = c.dim / c.group;
    if (c.dim == 128) {
        const RowArgs A = row_args<128>(c, ks, vs, n, start, n_tok);
        if (ng == 4) return rows_ng<128, 4>(A, type, read, k, v, st);
        if (ng == 2) return rows_ng<128, 2>(A, type, read, k, v, st);
        return rows_ng<128, 1>(A, type, read, k, v, st);
    }
    const RowArgs A = row_args<64>(c, ks, vs, n, start, n_tok);
    if (ng == 2) return rows_ng<64, 2>(A, type, read, k, v, st);
    return rows_ng<64, 1>(A, type, read, k, v, st);
}

}  // namespace

extern "C" cudaError_t kie_launch_kv4_append(const Kv4* c, const void* k, const void* v, const Kv4Strides* ks,
                                             const Kv4Strides* vs, int type, int n, const int32_t* start,
                                             const int32_t* n_tok, cudaStream_t st) {
    return rows(*c, const_cast<void*>(k), const_cast<void*>(v), *ks, *vs, type, false, n, start, n_tok, st);
}

extern "C" cudaError_t kie_launch_kv4_read(const Kv4* c, void* k, void* v, const Kv4Strides* ks, const Kv4Strides* vs,
                                           int type, int n, const int32_t* start, const int32_t* n_tok,
                                           cudaStream_t st) {
    return rows(*c, k, v, *ks, *vs, type, true, n, start, n_tok, st);
}

// Floats of workspace.  Stream form: a partial of CTA i for item k lies at slot k +
// i: a CTA's items and an item's CTAs are both consecutive, so no two (item, CTA)
// pairs that meet share a slot.  The cluster form needs none.
extern "C" size_t kie_kv4_attention_ws_floats(const Kv4Attn* a, int sms) {
    if (many_tokens(*a, sms)) return kie_kv4_chunk_ws_floats(a, sms);
    const Plan p = plan_of(*a, sms);
    return p.S ? 0 : size_t(p.items + p.nctas) * rows_of(p.mode) * (a->c.dim + 2);
}

extern "C" cudaError_t kie_launch_kv4_attention(const Kv4Attn* a, int sms, cudaStream_t st) {
    if (many_tokens(*a, sms)) return kie_launch_kv4_chunk(a, sms, st);
    const Plan p = plan_of(*a, sms);
    const AttnArgs A{*a, p.per, p.nrt, p.nctas};
    const int ng = a->c.dim / a->c.group;
    if (a->c.dim == 128) {
        if (ng == 4) return launch_attention_t<128, 4>(A, p, st);
        if (ng == 2) return launch_attention_t<128, 2>(A, p, st);
        return launch_attention_t<128, 1>(A, p, st);
    }
    if (ng == 2) return launch_attention_t<64, 2>(A, p, st);
    return launch_attention_t<64, 1>(A, p, st);
}
