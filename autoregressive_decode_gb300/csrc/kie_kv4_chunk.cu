// Attention of many new tokens (prompt chunks, long drafts) over the 4-bit K/V
// cache, on the 5th-generation tensor cores; see kie_kv4.cu for few tokens.
//
// One CTA takes 128 query rows (tokens x the query heads that share a K/V head) of
// one request and one stretch of the keys, two CTAs per SM, so that one's tensor
// work fills the other's softmax.  Per tile of 128 keys:
//   warps 4-7   thread = key: codes from global memory (a tile ahead, in registers)
//               to fp16 values code * s + z, rounded once, into the K and V tiles;
//   warp 4      also issues S = Q K^T and O += P V (tcgen05.mma, M 128), S and O in TMEM;
//   warps 0-3   thread = query row: running maximum, P = 2^(S - m) as fp16 over the
//               first half of S's columns, running sum; O is rescaled only when a
//               maximum grew by more than 2^8 (exact either way: m is any
//               reference, fp16 holds 2^15).
// Tiles use the canonical no-swizzle layouts, K as rows of channels (K-major), V as
// stored (MN-major).  Within 8 channels the order is 0 4 1 5 2 6 3 7, in which the
// nibbles of a word come apart; Q is stored alike and O's columns are read alike.
//
// The tensor pipe needs 1,024 cycles per tile and CTA; unpacking (2,100 warp
// instructions) and softmax (1,600) need about as many issue slots.
// Rounding: K, V and P to fp16 (2^-12 relative on average less), 16 times finer
// than the bf16 results this serves.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "kie_device.cuh"
#include "kie_kv4.h"

using namespace kie;

namespace {

constexpr int KEYS = 128;             // keys per tile
constexpr int ROWS = 128;             // query rows per CTA
constexpr int THREADS = 256;
constexpr int WAIT_TRIES = 100000;    // of up to 20 us each: 2 s, then the rows become NaN
constexpr float LAZY = 8.f;           // log2 of the growth of a maximum that is left alone
constexpr float UP = 7.f;             // p is at most 2^(LAZY + UP): fp16's range

struct ChunkArgs {
    Kv4Attn a;
    int32_t per, nrt, nsplit;
};

template <int D>
struct Sm {
    static constexpr uint32_t SBO = (D / 8) * 128;                       // 8 rows of a K-major tile (8 keys of V)
    static constexpr uint32_t TILE = 128 * D * 2;
    static constexpr uint32_t Q = 0, K = TILE, V = 2 * TILE, BARS = 3 * TILE;
    static constexpr uint32_t RAW = BARS + 128;
    // never three CTAs on an SM: TMEM holds two
    static constexpr uint32_t BYTES = RAW > 80 * 1024 ? RAW : 80 * 1024;
};
enum { KFULL = 0, KFREE, VFULL, VFREE, SFULL, PFULL, NBARS };

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* failed) {
    for (int i = 0; i < WAIT_TRIES; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 15 && *failed) return false;
    }
    *failed = 1;
    return false;
}

// A operand (P, fp16 pairs in 32-bit columns) from TMEM, B from shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// Four pairs of codes (nibbles n of the word's halves) to code * s + z, rounded once.
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t s2, uint32_t z2) {
    constexpr uint32_t K1024 = 0x64006400u, M1024 = 0xE400E400u;      // fp16 1024 + code, -1024
    constexpr uint32_t SIXTEENTH = 0x2C002C00u, M64 = 0xD400D400u;    // 1/16, -64
    const uint32_t w8 = w >> 8;
    uint4 r;
    r.x = hfma2(hadd2((w & 0x000F000Fu) | K1024, M1024), s2, z2);
    r.y = hfma2(hfma2((w & 0x00F000F0u) | K1024, SIXTEENTH, M64), s2, z2);
    r.z = hfma2(hadd2((w8 & 0x000F000Fu) | K1024, M1024), s2, z2);
    r.w = hfma2(hfma2((w8 & 0x00F000F0u) | K1024, SIXTEENTH, M64), s2, z2);
    return r;
}

template <int T> struct El;
template <> struct El<KV4_BF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};

// One key's codes and parameters, as loaded.
template <int D, int NG>
struct Raw {
    uint4 c[4];                       // D == 64: two of them
    uint32_t p[NG == 4 ? 8 : NG == 2 ? 4 : 2];   // K: the position's words; V: the pair's
};

template <int D, int NG, int T>
__global__ void __launch_bounds__(THREADS, 2) kv4_chunk_kernel(const ChunkArgs A) {
    using E = typename El<T>::type;
    using L = Sm<D>;
    constexpr int BLK = D / 32, BPG = BLK / NG, NC = D / 32;      // 16-byte loads of a key's codes
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint32_t* taddr = reinterpret_cast<uint32_t*>(bar + NBARS);
    volatile int* failed = reinterpret_cast<volatile int*>(taddr + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Kv4& c = A.a.c;

    // later row tiles see more keys: they go first
    const int split = int(blockIdx.x) % A.nsplit, item = int(blockIdx.x) / A.nsplit;
    const int bh = item % (c.batch * c.heads), rt = A.nrt - 1 - item / (c.batch * c.heads);
    const int b = bh / c.heads, head = bh % c.heads, r0 = rt * ROWS;
    const int len = min(max(__ldg(A.a.kv_len + b), 0), c.max_ctx);
    const int n_new = A.a.n_tok ? min(max(__ldg(A.a.n_tok + b), 0), A.a.n_q) : A.a.n_q;
    const int rows = n_new * A.per;
    if (r0 >= rows) return;
    int lo = 0, hi = len;
    if (A.a.causal) {
        const int t0 = r0 / A.per, t1 = (min(r0 + ROWS, rows) - 1) / A.per;
        hi = max(0, len - n_new + t1 + 1);
        if (A.a.window > 0) lo = max(0, len - n_new + t0 + 1 - A.a.window);
        if (lo >= hi) lo = hi = 0;
    }
    const int all = hi > lo ? (hi + KEYS - 1) / KEYS - lo / KEYS : 0;
    const int first = int(int64_t(all) * split / A.nsplit), ntile = int(int64_t(all) * (split + 1) / A.nsplit) - first;
    const int base = (lo / KEYS + first) * KEYS;

    if (tid == 0) {
        mbar_init(&bar[KFULL], 4);
        mbar_init(&bar[KFREE], 1);
        mbar_init(&bar[VFULL], 4);
        mbar_init(&bar[VFREE], 1);
        mbar_init(&bar[SFULL], 1);
        mbar_init(&bar[PFULL], 4);
        *failed = 0;
        mbar_fence_init();
    }
    if (warp == 4) tmem_alloc(taddr, 256);

    // ---- Q: thread = row; a power of two brings the row's largest element to [1, 2)
    const int r = r0 + tid;                        // warps 0-3
    const bool have = tid < ROWS && r < rows;
    const int tok = have ? r / A.per : 0, hq = head * A.per + (have ? r - tok * A.per : 0);
    float cq = 0.f;                                // from S to log2 units
    if (warp < 4) {
        const E* q = static_cast<const E*>(A.a.q) + b * A.a.qs.b + tok * A.a.qs.t + hq * A.a.qs.h;
        const bool vec = (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
        auto load = [&](int i) {
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (have) {
                if (vec) raw = __ldg(reinterpret_cast<const uint4*>(q) + i);
                else {
                    E* e = reinterpret_cast<E*>(&raw);
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = q[i * 8 + j];
                }
            }
            return raw;
        };
        float mx = 0.f;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
            const uint4 raw = load(i);
            const E* e = reinterpret_cast<const E*>(&raw);
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(El<T>::to(e[j])));
        }
        const int ex = min(max(((__float_as_int(mx) >> 23) & 255) - 127, -100), 114);
        const float up = copysignf(__int_as_float((127 - ex) << 23), A.a.scale);
        cq = fmaxf(fabsf(A.a.scale) * 1.4426950408889634f * __int_as_float((127 + ex) << 23), 1.2e-38f);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
            const uint4 raw = load(i);         // from L1
            const E* e = reinterpret_cast<const E*>(&raw);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = El<T>::to(e[j]) * up;
            *reinterpret_cast<uint4*>(sm + L::Q + (tid >> 3) * L::SBO + i * 128 + (tid & 7) * 16) =
                make_uint4(pack_h2(f[0], f[4]), pack_h2(f[1], f[5]), pack_h2(f[2], f[6]), pack_h2(f[3], f[7]));
        }
        fence_proxy_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = *taddr, tO = tS + 128u;

    if (warp >= 4) {
        // ---- codes to tiles: thread = key
        const int k = tid - 128;
        const size_t row0 = (size_t(b) * c.heads + head) * c.ctx_pad;
        auto load = [&](int i, Raw<D, NG>& K, Raw<D, NG>& V) {
            const int p = min(base + i * KEYS + k, c.ctx_pad - 1);   // in the head's memory; zeroed below where not stored
            const uint4* kc = reinterpret_cast<const uint4*>(c.kc + (row0 + p) * (D / 2));
            const uint4* vc = reinterpret_cast<const uint4*>(c.vc + (row0 + p) * (D / 2));
#pragma unroll
            for (int j = 0; j < NC; ++j) { K.c[j] = __ldg(kc + j); V.c[j] = __ldg(vc + j); }
            const uint32_t* kp = reinterpret_cast<const uint32_t*>(c.kp) + (row0 + p) * NG;
            const int rr = p & 7, t = rr >> 2 ? 7 - rr : rr;
            const uint32_t* vp = reinterpret_cast<const uint32_t*>(c.vp) + ((row0 + p) >> 3) * (8 * NG) + t * 2 * NG;
#pragma unroll
            for (int j = 0; j < NG; ++j) K.p[j] = __ldg(kp + j);
#pragma unroll
            for (int j = 0; j < 2 * NG; ++j) V.p[j] = __ldg(vp + j);
        };
        Raw<D, NG> K, V;
        constexpr uint32_t IS = (1u << 4) | (uint32_t(KEYS >> 3) << 17) | (uint32_t(ROWS >> 4) << 24);
        constexpr uint32_t IO = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(ROWS >> 4) << 24);
        const bool issuer = tid == 128;
        int issued_s = 0, issued = 0;
        if (ntile > 0) load(0, K, V);
        for (int i = 0; i < ntile; ++i) {
            const int p = base + i * KEYS + k;
            const bool stored = p < len;
            const uint32_t ph = uint32_t(i) & 1u;
            if (__any_sync(0xffffffffu, i > 0 && !wait_for(&bar[KFREE], ph ^ 1u, failed))) break;
            uint8_t* dst = sm + L::K + (k >> 3) * L::SBO + (k & 7) * 16;
#pragma unroll
            for (int bl = 0; bl < BLK; ++bl) {
                // scale and zero of the block's group, doubled
                const int gi = bl / BPG;
                const uint32_t sw = NG == 1 ? K.p[0] : K.p[gi >> 1], zw = NG == 1 ? K.p[0] : K.p[NG / 2 + (gi >> 1)];
                const uint32_t s2 = stored ? __byte_perm(sw, 0u, (NG > 1 && (gi & 1)) ? 0x3232 : 0x1010) : 0u;
                const uint32_t z2 = stored ? __byte_perm(zw, 0u, (NG == 1 || (gi & 1)) ? 0x3232 : 0x1010) : 0u;
                // word t * BLK + bl of the key: channels 32 bl + 8 t ..
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int wi = t * BLK + bl;
                    const uint4& q = K.c[wi >> 2];
                    const uint32_t w = (wi & 3) == 0 ? q.x : (wi & 3) == 1 ? q.y : (wi & 3) == 2 ? q.z : q.w;
                    *reinterpret_cast<uint4*>(dst + (bl * 4 + t) * 128) = values8(w, s2, z2);
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[KFULL]);
            // S overlies P and V is read by the same product: the last one has to be done
            bool ok = i == 0 || wait_for(&bar[VFREE], ph ^ 1u, failed);
            if (issuer && ok && (ok = wait_for(&bar[KFULL], ph, failed))) {
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_f16(tS, smem_desc_noswz(sm + L::Q + kk * 256, 128, L::SBO), smem_desc_noswz(sm + L::K + kk * 256, 128, L::SBO),
                               IS, kk != 0 ? 1u : 0u);
                tc_commit(&bar[SFULL]);
                tc_commit(&bar[KFREE]);
                issued_s = i + 1;
            }
            if (__any_sync(0xffffffffu, !ok)) break;
            dst = sm + L::V + (k >> 3) * L::SBO + (k & 7) * 16;
            const uint32_t half = (p & 4) ? 0x3232u : 0x1010u;         // this position of its pair
#pragma unroll
            for (int bl = 0; bl < BLK; ++bl) {
                const int gi = bl / BPG;
                const uint32_t s2 = stored ? __byte_perm(V.p[gi], 0u, half) : 0u;
                const uint32_t z2 = stored ? __byte_perm(V.p[NG + gi], 0u, half) : 0u;
                // units 2 i2 and 2 i2 + 1 of the block: channels 32 bl + 8 i2 ..
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) {
                    const int u0 = 2 * i2 * BLK + bl, u1 = u0 + BLK;     // 16-bit units
                    auto word = [&](int u) {
                        const int wi = u >> 1;
                        const uint4& q = V.c[wi >> 2];
                        return (wi & 3) == 0 ? q.x : (wi & 3) == 1 ? q.y : (wi & 3) == 2 ? q.z : q.w;
                    };
                    const uint32_t w = __byte_perm(word(u0), word(u1), (u0 & 1) ? 0x7632 : 0x5410);
                    *reinterpret_cast<uint4*>(dst + (bl * 4 + i2) * 128) = values8(w, s2, z2);
                }
            }
            if (i + 1 < ntile) load(i + 1, K, V);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[VFULL]);
            if (issuer && (ok = wait_for(&bar[VFULL], ph, failed) && wait_for(&bar[PFULL], ph, failed))) {
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < KEYS / 16; ++kk)
                    mma_ts(tO, tS + kk * 8, smem_desc_noswz(sm + L::V + kk * 2 * L::SBO, L::SBO, 128), IO, (i > 0 || kk > 0) ? 1u : 0u);
                tc_commit(&bar[VFREE]);
                issued = i + 1;
            }
            if (__any_sync(0xffffffffu, !ok)) break;
        }
        // every product has landed before the accumulators are read or given back
        if (issuer && issued_s > issued) wait_for(&bar[KFREE], uint32_t(issued_s - 1) & 1u, failed);
        if (issuer && issued) wait_for(&bar[VFREE], uint32_t(issued - 1) & 1u, failed);
        __syncwarp();
    }
    float m = -INFINITY, l = 0.f;
    const uint32_t my = uint32_t(warp * 32) << 16;       // this warp's TMEM lanes
    if (warp < 4) {
        // ---- softmax: thread = row
        const int last = !have ? -1 : A.a.causal ? len - n_new + tok : len - 1;
        const int firstk = A.a.window > 0 ? last - A.a.window + 1 : 0;
        const int all_lo = __reduce_max_sync(0xffffffffu, have ? firstk : 0);
        const int all_hi = __reduce_min_sync(0xffffffffu, have ? last : 1 << 30);
        for (int i = 0; i < ntile; ++i) {
            if (__any_sync(0xffffffffu, !wait_for(&bar[SFULL], uint32_t(i) & 1u, failed))) break;
            tc_fence_after();
            const int p0 = base + i * KEYS;
            const bool edge = p0 < all_lo || p0 + KEYS - 1 > all_hi;      // uniform over the warp
            float mt = -INFINITY;
#pragma unroll
            for (int c0 = 0; c0 < KEYS; c0 += 32) {
                uint32_t s[32];
                tmem_ld_32x32b_x32(tS + my + c0, s);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (p0 + c0 + e < firstk || p0 + c0 + e > last) s[e] = 0xFF800000u;
                }
                float a = __uint_as_float(s[0]), b2 = __uint_as_float(s[1]);
#pragma unroll
                for (int e = 2; e < 32; e += 2) { a = max_nan(a, __uint_as_float(s[e])); b2 = max_nan(b2, __uint_as_float(s[e + 1])); }
                mt = max_nan(mt, max_nan(a, b2));
            }
            mt *= cq;
            float f = 1.f;
            if (!(mt <= m + LAZY)) {            // also at the first keys and for a NaN
                f = m == -INFINITY ? 0.f : ex2(m - mt);
                l *= f;
                m = mt;
            }
            if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(tO + my + c0, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st_32x32b_x32(tO + my + c0, o);
                }
            }
            const float ref = (m == -INFINITY ? 0.f : m) - UP;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c0 = 0; c0 < KEYS; c0 += 32) {
                uint32_t s[32], h[16];
                tmem_ld_32x32b_x32(tS + my + c0, s);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (p0 + c0 + e < firstk || p0 + c0 + e > last) s[e] = 0xFF800000u;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                                make_float2(cq, cq), make_float2(-ref, -ref));
                    const float2 p = make_float2(ex2(x.x), ex2(x.y));
                    sum = __fadd2_rn(sum, p);
                    h[e] = pack_h2(p.x, p.y);
                }
                tmem_st_x16(tS + my + c0 / 2, h);     // columns of S that are read already
            }
            l += sum.x + sum.y;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[PFULL]);
        }
    }
    __syncthreads();                   // warp 4 has waited for the last product
    tc_fence_after();
    if (warp < 4) {
        const bool bad = *failed != 0;
        float* part = A.nsplit > 1 ? A.a.ws + (size_t(item) * A.nsplit + split) * (ROWS * (D + 2)) : nullptr;
        E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + tok * A.a.os.t + hq * A.a.os.h;
        const bool vec = (reinterpret_cast<uintptr_t>(op) & 15u) == 0;
        const float il = bad ? __int_as_float(0x7FC00000) : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            if (ntile > 0) tmem_ld_32x32b_x32(tO + my + c0, o);
            else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
            if (!have) continue;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                // columns 0 .. 7 are channels 0 4 1 5 2 6 3 7
                const int at[8] = {0, 2, 4, 6, 1, 3, 5, 7};
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(o[e + at[j]]);
                if (A.nsplit > 1) {
#pragma unroll
                    for (int j = 0; j < 8; j += 4)
                        *reinterpret_cast<float4*>(part + size_t(tid) * D + c0 + e + j) =
                            bad ? make_float4(il, il, il, il) : make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                } else {
                    uint4 w;
                    E* we = reinterpret_cast<E*>(&w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) we[j] = El<T>::from(l == 0.f && !bad ? 0.f : v[j] * il);
                    if (vec) *reinterpret_cast<uint4*>(op + c0 + e) = w;
                    else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) op[c0 + e + j] = we[j];
                    }
                }
            }
        }
        if (A.nsplit > 1 && have) *reinterpret_cast<float2*>(part + ROWS * D + 2 * tid) = make_float2(m, l);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) tmem_dealloc(tS, 256);
}

// Join the stretches of the keys.  One block per item and 2 rows (D = 128) or 4.
template <int D, int T>
__global__ void __launch_bounds__(256) kv4_chunk_join_kernel(const ChunkArgs A) {
    using E = typename El<T>::type;
    constexpr int PER = ROWS * D / 256;
    const Kv4& c = A.a.c;
    const int item = int(blockIdx.x) / PER, i = int(blockIdx.x) % PER * 256 + threadIdx.x;
    const int bh = item % (c.batch * c.heads), rt = A.nrt - 1 - item / (c.batch * c.heads);
    const int b = bh / c.heads, head = bh % c.heads, row = rt * ROWS + i / D;
    const int n_new = A.a.n_tok ? min(max(__ldg(A.a.n_tok + b), 0), A.a.n_q) : A.a.n_q;
    if (row >= n_new * A.per) return;
    const float* part = A.a.ws + size_t(item) * A.nsplit * (ROWS * (D + 2));
    float M = -INFINITY, l = 0.f, o = 0.f;
    for (int k = 0; k < A.nsplit; ++k) {
        const float* p = part + size_t(k) * (ROWS * (D + 2));
        const float2 ml = *reinterpret_cast<const float2*>(p + ROWS * D + 2 * (i / D));
        if (ml.x == -INFINITY) continue;
        const float mn = max_nan(M, ml.x), f0 = M == -INFINITY ? 0.f : ex2(M - mn), f1 = ex2(ml.x - mn);
        l = l * f0 + ml.y * f1;
        o = o * f0 + p[i] * f1;
        M = mn;
    }
    const int tok = row / A.per;
    E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + tok * A.a.os.t + (head * A.per + row - tok * A.per) * A.a.os.h;
    op[i % D] = El<T>::from(l == 0.f ? 0.f : o / l);
}

template <int D, int NG, int T>
cudaError_t launch(const ChunkArgs& A, int items, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(done.load(std::memory_order_acquire) & bit)) {
        r = cudaFuncSetAttribute(kv4_chunk_kernel<D, NG, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm<D>::BYTES);
        if (r != cudaSuccess) return r;
        if (dev < 64) done.fetch_or(bit, std::memory_order_release);
    }
    kv4_chunk_kernel<D, NG, T><<<unsigned(items) * A.nsplit, THREADS, Sm<D>::BYTES, st>>>(A);
    r = cudaGetLastError();
    if (r != cudaSuccess || A.nsplit == 1) return r;
    kv4_chunk_join_kernel<D, T><<<unsigned(items) * (ROWS * D / 256), 256, 0, st>>>(A);
    return cudaGetLastError();
}

struct ChunkPlan { int per, nrt, nsplit; int64_t items; };
ChunkPlan plan_of(const Kv4Attn& a, int sms) {
    ChunkPlan p;
    p.per = a.heads / a.c.heads;
    p.nrt = int((int64_t(a.n_q) * p.per + ROWS - 1) / ROWS);
    p.items = int64_t(p.nrt) * a.c.batch * a.c.heads;
    int64_t keys = a.c.max_ctx;
    if (a.window > 0) keys = std::min<int64_t>(keys, int64_t(a.window) + ROWS / p.per + 1);
    const int64_t tiles = (keys + KEYS - 1) / KEYS + (a.window > 0);
    // stretches of at least four tiles until two CTAs per SM are busy
    p.nsplit = int(std::max<int64_t>(1, std::min<int64_t>(2 * sms / std::max<int64_t>(p.items, 1), tiles / 4)));
    return p;
}

}  // namespace

extern "C" size_t kie_kv4_chunk_ws_floats(const Kv4Attn* a, int sms) {
    const ChunkPlan p = plan_of(*a, sms);
    return p.nsplit > 1 ? size_t(p.items) * p.nsplit * (ROWS * (a->c.dim + 2)) : 0;
}

extern "C" cudaError_t kie_launch_kv4_chunk(const Kv4Attn* a, int sms, cudaStream_t st) {
    const ChunkPlan p = plan_of(*a, sms);
    const ChunkArgs A{*a, p.per, p.nrt, p.nsplit};
    const int ng = a->c.dim / a->c.group, items = int(p.items);
    if (a->c.dim == 128) {
        if (ng == 4) return launch<128, 4, KV4_BF16>(A, items, st);
        if (ng == 2) return launch<128, 2, KV4_BF16>(A, items, st);
        return launch<128, 1, KV4_BF16>(A, items, st);
    }
    if (ng == 2) return launch<64, 2, KV4_BF16>(A, items, st);
    return launch<64, 1, KV4_BF16>(A, items, st);
}
