// Attention of many new tokens (prompt chunks, long drafts) over the 4-bit K/V
// cache, on the 5th-generation tensor cores; see kie_kv4.cu for few tokens.
//
// One CTA takes two tiles of 128 query rows (tokens x the query heads that share a
// K/V head) of one request and one stretch of the keys, in tiles of 128 keys:
//   warps 16-19  thread = key: codes from global memory (a tile ahead, in registers)
//                to fp16 values code * s + z, rounded once, into K and V tiles, two
//                of each in flight, shared by both row tiles;
//   warp 20      issues S = Q K^T and O += P V (tcgen05.mma, M 128), 64 keys at a
//                time, S and O in TMEM;
//   warps 0-15   two threads per query row, 32 of the 64 keys each: running maximum,
//                P = 2^(S - m) as fp16 over half of its S columns, running sum; O is
//                rescaled only when a maximum grew by more than 2^8 (exact either way:
//                m is any reference, and fp16 holds 2^15).
// Of a row tile's two S buffers one is worked on while the next S is computed into the
// other, once the product that read P there is done (the order of two tcgen05.mma with
// different accumulators is not guaranteed otherwise).
// Tiles use the canonical no-swizzle layouts, K as rows of channels (K-major), V as
// stored (MN-major); the pipe runs them at its full rate (64 cycles an instruction).
// Within 8 channels the order is 0 4 1 5 2 6 3 7, in which the nibbles of a word come
// apart; Q is stored alike and O's columns are read alike.
//
// Rounding: K, V and P to fp16 (2^-12 relative on average less), 16 times finer
// than the bf16 results this serves.
//
// 1,024 tokens x 32 heads of 128 at the end of 4,096 keys (60 GFLOP): 89 us, 0.67 PFLOP/s.
// The matrix unit's own time there is 45 us (51 cycles an instruction for S, 65 for P V), 68
// us with everything else taken out of the loop but its barriers; the softmax shares the SM
// with the conversion of the codes.  A sixth of the SMs is idle: 128 CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "kie_device.cuh"
#include "kie_kv4.h"

using namespace kie;

namespace {

constexpr int KEYS = 128;             // keys per K and V tile
constexpr int STEP = 64;              // keys per S
constexpr int ROWS = 256;             // query rows per CTA, in two tiles
constexpr int THREADS = 672;
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
    static constexpr uint32_t Q = 0, K = 2 * TILE, V = 4 * TILE, BARS = 6 * TILE;
    static constexpr uint32_t MAXES = BARS + 256;                        // [parity][row tile][half][128]
    static constexpr uint32_t SUMS = MAXES + 2 * 2 * 2 * 128 * 4;        // [row tile][half][128]
    static constexpr uint32_t USED = SUMS + 2 * 2 * 128 * 4;
    // never two CTAs on an SM: one takes all of TMEM
    static constexpr uint32_t BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
};
// K, V: per stage; S, P: per row tile and buffer (each may be a step ahead of who waits
// for it, and a barrier tells only two phases apart); PVDONE: per row tile.
enum { KFULL = 0, KFREE = 2, VFULL = 4, VFREE = 6, SFULL = 8, PFULL = 12, PVDONE = 16, FIN = 18, NBARS = 19 };

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* failed) {
#pragma unroll 1
    for (int i = 0; i < WAIT_TRIES; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 15 && *failed) return false;
    }
    *failed = 1;
    return false;
}

// The tensor instructions are issued by whole warps under a predicate that one lane
// holds: their descriptors then stay in uniform registers (a branch to one thread
// costs a transfer per operand, 150 cycles an instruction beside four busy warps).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p;
}
// D[tmem] (+)= A B^T, A and B from shared memory; descriptors by their low words and a
// common high one.
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t el) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(el), "n"(ACC ? 1 : 0)
        : "memory");
}
// A (P, fp16 pairs in 32-bit columns) from TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t accumulate,
                                       uint32_t el) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.u32 q, %6, 0;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate), "r"(el)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t el) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(el)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 16 columns of this warp's TMEM lanes without waiting; and the wait for every load,
// through which the registers go, so that no use of them moves before it.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
        :: "memory");
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
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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

// Whether code 15 of either group reaches beyond fp16 (where values as large as the type has
// were stored and s was rounded up): an exponent of all ones in 15 s + z.
__device__ __forceinline__ uint32_t beyond(uint32_t s2, uint32_t z2) {
    return ((hfma2(0x4B804B80u, s2, z2) & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
// Keeps a key's values inside the type.
template <int D>
__device__ __forceinline__ void inside(uint8_t* dst) {
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {
        uint32_t* const w = reinterpret_cast<uint32_t*>(dst + i * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("min.f16x2 %0, %0, %1;" : "+r"(w[j]) : "r"(0x7BFF7BFFu));
    }
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
__global__ void __launch_bounds__(THREADS, 1) kv4_chunk_kernel(const ChunkArgs A) {
    using E = typename El<T>::type;
    using L = Sm<D>;
    constexpr int BLK = D / 32, BPG = BLK / NG, NC = D / 32;      // NC: 16-byte loads of a key's codes
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint32_t* taddr = reinterpret_cast<uint32_t*>(bar + NBARS);
    volatile int* failed = reinterpret_cast<volatile int*>(taddr + 1);
    float* maxes = reinterpret_cast<float*>(sm + L::MAXES);
    float* sums = reinterpret_cast<float*>(sm + L::SUMS);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // uniform to the compiler
    const Kv4& c = A.a.c;

    // later row tiles see more keys: they go first
    const int split = int(blockIdx.x) % A.nsplit, item = int(blockIdx.x) / A.nsplit;
    const int bh = item % (c.batch * c.heads), rt = A.nrt - 1 - item / (c.batch * c.heads);
    const int b = bh / c.heads, head = bh % c.heads, r0 = rt * ROWS;
    const int len = min(max(__ldg(A.a.kv_len + b), 0), c.max_ctx);
    const int n_new = A.a.n_tok ? min(max(__ldg(A.a.n_tok + b), 0), A.a.n_q) : A.a.n_q;
    const int rows = n_new * A.per;
    if (r0 >= rows) return;
    const int ntl = r0 + 128 < rows ? 2 : 1;       // row tiles with rows
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[KFULL + i], 4);
            mbar_init(&bar[KFREE + i], 1);
            mbar_init(&bar[VFULL + i], 4);
            mbar_init(&bar[VFREE + i], 1);
            mbar_init(&bar[PVDONE + i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar[SFULL + i], 1);
            mbar_init(&bar[PFULL + i], 8);
        }
        mbar_init(&bar[FIN], 1);
        *failed = 0;
        mbar_fence_init();
    }
    if (warp == 20) tmem_alloc(taddr, 512);

    // ---- Q: a power of two brings a row's largest element to [1, 2)
    // softmax thread: row tile t, half h of the keys, row `lr` of the tile
    const int t = warp >> 3, h = (warp >> 2) & 1, lr = (warp & 3) * 32 + lane;
    const int r = r0 + t * 128 + lr;
    const bool have = warp < 16 && r < rows;
    const int tok = have ? r / A.per : 0, hq = head * A.per + (have ? r - tok * A.per : 0);
    float cq = 0.f;                                // from S to log2 units
    if (warp < 16) {
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
        uint8_t* dst = sm + L::Q + t * L::TILE + (lr >> 3) * L::SBO + (lr & 7) * 16;
#pragma unroll 4
        for (int i = h * (D / 16); i < (h + 1) * (D / 16); ++i) {        // this half's channels, from L1
            const uint4 raw = load(i);
            const E* e = reinterpret_cast<const E*>(&raw);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = El<T>::to(e[j]) * up;
            *reinterpret_cast<uint4*>(dst + i * 128) =
                make_uint4(pack_h2(f[0], f[4]), pack_h2(f[1], f[5]), pack_h2(f[2], f[6]), pack_h2(f[3], f[7]));
        }
        fence_proxy_async_shared();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *taddr;                  // S of the row tiles at 0 and 128, O at 256 and 384

    float m = -INFINITY, l = 0.f;
    auto ready = [&](int bi, uint32_t ph) { return !__any_sync(0xffffffffu, !wait_for(&bar[bi], ph, failed)); };
    if (warp >= 16 && warp < 20) {
        // ---- codes to tiles: thread = key
        const int k = tid - 512;
        const size_t row0 = (size_t(b) * c.heads + head) * c.ctx_pad;
        Raw<D, NG> K, V;
        auto load_k = [&](int i) {
            const int p = min(base + i * KEYS + k, c.ctx_pad - 1);   // in the head's memory; zeroed below where not stored
            const uint4* kc = reinterpret_cast<const uint4*>(c.kc + (row0 + p) * (D / 2));
            const uint32_t* kp = reinterpret_cast<const uint32_t*>(c.kp) + (row0 + p) * NG;
#pragma unroll
            for (int j = 0; j < NC; ++j) K.c[j] = __ldg(kc + j);
#pragma unroll
            for (int j = 0; j < NG; ++j) K.p[j] = __ldg(kp + j);
        };
        auto load_v = [&](int i) {
            const int p = min(base + i * KEYS + k, c.ctx_pad - 1);
            const uint4* vc = reinterpret_cast<const uint4*>(c.vc + (row0 + p) * (D / 2));
            const int rr = p & 7, pt = rr >> 2 ? 7 - rr : rr;
            const uint32_t* vp = reinterpret_cast<const uint32_t*>(c.vp) + ((row0 + p) >> 3) * (8 * NG) + pt * 2 * NG;
#pragma unroll
            for (int j = 0; j < NC; ++j) V.c[j] = __ldg(vc + j);
#pragma unroll
            for (int j = 0; j < 2 * NG; ++j) V.p[j] = __ldg(vp + j);
        };
        const uint32_t at = (k >> 3) * L::SBO + (k & 7) * 16;
        auto put_k = [&](int i) {
            const bool stored = base + i * KEYS + k < len;
            uint8_t* dst = sm + L::K + (i & 1) * L::TILE + at;
#pragma unroll
            for (int bl = 0; bl < BLK; ++bl) {
                // scale and zero of the block's group, doubled
                const int gi = bl / BPG;
                const uint32_t sw = NG == 1 ? K.p[0] : K.p[gi >> 1], zw = NG == 1 ? K.p[0] : K.p[NG / 2 + (gi >> 1)];
                const uint32_t s2 = stored ? __byte_perm(sw, 0u, (NG > 1 && (gi & 1)) ? 0x3232 : 0x1010) : 0u;
                const uint32_t z2 = stored ? __byte_perm(zw, 0u, (NG == 1 || (gi & 1)) ? 0x3232 : 0x1010) : 0u;
                // word j * BLK + bl of the key: channels 32 bl + 8 j ..
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int wi = j * BLK + bl;
                    const uint4& q = K.c[wi >> 2];
                    const uint32_t w = (wi & 3) == 0 ? q.x : (wi & 3) == 1 ? q.y : (wi & 3) == 2 ? q.z : q.w;
                    *reinterpret_cast<uint4*>(dst + (bl * 4 + j) * 128) = values8(w, s2, z2);
                }
            }
            uint32_t wide = NG == 1 ? K.p[0] & 0xFFFFu : 0u;            // a scale of 2 or more: look closer
#pragma unroll
            for (int gi = 0; gi < NG / 2; ++gi) wide |= K.p[gi];
            if (__any_sync(0xffffffffu, wide & 0x40004000u)) {
                uint32_t far = NG == 1 ? beyond(K.p[0], K.p[0] >> 16) & 0xFFFFu : 0u;
#pragma unroll
                for (int gi = 0; gi < NG / 2; ++gi) far |= beyond(K.p[gi], K.p[NG / 2 + gi]);
                if (far) inside<D>(dst);
            }
        };
        auto put_v = [&](int i) {
            const int p = base + i * KEYS + k;
            const bool stored = p < len;
            const uint32_t half = (p & 4) ? 0x3232u : 0x1010u;       // this position of its pair, doubled
            uint8_t* dst = sm + L::V + (i & 1) * L::TILE + at;
#pragma unroll
            for (int bl = 0; bl < BLK; ++bl) {
                const int gi = bl / BPG;
                const uint32_t s2 = stored ? __byte_perm(V.p[gi], 0u, half) : 0u;
                const uint32_t z2 = stored ? __byte_perm(V.p[NG + gi], 0u, half) : 0u;
                // units 2 j and 2 j + 1 of the block: channels 32 bl + 8 j ..
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u0 = 2 * j * BLK + bl, u1 = u0 + BLK;     // 16-bit units
                    auto word = [&](int u) {
                        const int wi = u >> 1;
                        const uint4& q = V.c[wi >> 2];
                        return (wi & 3) == 0 ? q.x : (wi & 3) == 1 ? q.y : (wi & 3) == 2 ? q.z : q.w;
                    };
                    const uint32_t w = __byte_perm(word(u0), word(u1), (u0 & 1) ? 0x7632 : 0x5410);
                    *reinterpret_cast<uint4*>(dst + (bl * 4 + j) * 128) = values8(w, s2, z2);
                }
            }
            uint32_t wide = 0u;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) wide |= V.p[gi];
            if (__any_sync(0xffffffffu, wide & 0x40004000u)) {
                uint32_t far = 0u;
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) far |= beyond(V.p[gi], V.p[NG + gi]);
                if (far) inside<D>(dst);
            }
        };
        // the tile that used the same stage last is done with it: its parity
        auto free_ph = [](int i) { return uint32_t((i >> 1) - 1) & 1u; };
        auto arrive = [&](int bi) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[bi]);
        };
        if (ntile > 0) {
            load_k(0);
            load_v(0);
            put_k(0);
            arrive(KFULL);
            if (ntile > 1) load_k(1);
        }
        for (int i = 0; i < ntile; ++i) {      // K runs a tile ahead of V
            if (i + 1 < ntile) {
                if (__any_sync(0xffffffffu, i > 0 && !wait_for(&bar[KFREE + ((i + 1) & 1)], free_ph(i + 1), failed))) break;
                put_k(i + 1);
                arrive(KFULL + ((i + 1) & 1));
                if (i + 2 < ntile) load_k(i + 2);
            }
            if (__any_sync(0xffffffffu, i > 1 && !wait_for(&bar[VFREE + (i & 1)], free_ph(i), failed))) break;
            put_v(i);
            arrive(VFULL + (i & 1));
            if (i + 1 < ntile) load_v(i + 1);
        }
    } else if (warp == 20) {
        // ---- the tensor cores
        const uint32_t el = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t IS = (1u << 4) | (uint32_t(STEP >> 3) << 17) | (uint32_t(128 >> 4) << 24);
        constexpr uint32_t IO = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);
        constexpr uint32_t HALF = STEP / 8 * (L::SBO / 16), STAGE = L::TILE / 16;       // addresses in units of 16 bytes
        const uint64_t dq = smem_desc_noswz(sm + L::Q, 128, L::SBO);
        const uint64_t dk = smem_desc_noswz(sm + L::K, 128, L::SBO), dv = smem_desc_noswz(sm + L::V, L::SBO, 128);
        // Nothing here branches on what one thread alone knows: a wait that runs out leaves
        // its mark in `failed` and the work goes on with what is there (the rows become NaN),
        // so that loops, descriptors and addresses stay in the uniform registers.
        const int nstep = __shfl_sync(0xffffffffu, 2 * ntile, 0), nt2 = __shfl_sync(0xffffffffu, ntl, 0);
        const uint32_t qlo = uint32_t(dq), klo = uint32_t(dk), vlo = uint32_t(dv);
        const uint32_t qhi = uint32_t(dq >> 32), vhi = uint32_t(dv >> 32);      // K's is Q's
        auto wait = [&](int bi, uint32_t parity) {
            wait_for(&bar[bi], parity, failed);
            __syncwarp();
        };
        // Steps j = 4 n + q: q alone gives the stage (q >> 1), the half of the key tile and
        // the S buffer (q & 1) and the parities of a buffer's and of a row tile's barriers;
        // `par` is that of the stages' barriers for n.  S of row tile tl and step q (up to
        // two steps ahead, q < 6):
        auto issue_s = [&](int tl, int q, uint32_t par) {
            if (tl == 0 && (q & 1) == 0) wait(KFULL + ((q >> 1) & 1), par ^ uint32_t(q >> 2));
            tc_fence_after();
            const uint32_t a = qlo + tl * STAGE, k = klo + ((q >> 1) & 1) * STAGE + (q & 1) * HALF;
            const uint32_t d = tm + tl * 128 + (q & 1) * STEP;
            mma_ss<false>(d, a, k, qhi, IS, el);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) mma_ss<true>(d, a + kk * 16, k + kk * 16, qhi, IS, el);
            commit(&bar[SFULL + 2 * tl + (q & 1)], el);
            if ((q & 1) && tl == nt2 - 1) commit(&bar[KFREE + ((q >> 1) & 1)], el);
        };
        auto issue_pv = [&](int tl, int q, uint32_t par, uint32_t accumulate) {
            if (tl == 0 && (q & 1) == 0) wait(VFULL + ((q >> 1) & 1), par);
            wait(PFULL + 2 * tl + (q & 1), uint32_t(q >> 1) & 1u);
            tc_fence_after();
            const uint32_t v = vlo + ((q >> 1) & 1) * STAGE + (q & 1) * HALF;
            const uint32_t p = tm + tl * 128 + (q & 1) * STEP, d = tm + 256 + tl * 128;
            mma_ts(d, p, v, vhi, IO, accumulate, el);
#pragma unroll
            for (int kk = 1; kk < STEP / 16; ++kk)
                mma_ts(d, p + (kk >> 1) * 32 + (kk & 1) * 8, v + kk * (2 * L::SBO / 16), vhi, IO, 1u, el);
            commit(&bar[PVDONE + tl], el);
            if ((q & 1) && tl == nt2 - 1) commit(&bar[VFREE + ((q >> 1) & 1)], el);
        };
        // A row tile's next S but one goes into the buffer whose P its last product has
        // read; with two row tiles the other one's work lies between the two.
        if (nstep > 0) {
            issue_s(0, 0, 0u);
            if (nt2 == 2) issue_s(1, 0, 0u);
            issue_s(0, 1, 0u);
        }
#pragma unroll 1
        for (int j0 = 0; j0 < nstep; j0 += 4) {
            const uint32_t par = uint32_t(j0 >> 2) & 1u;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = j0 + q;
                if (j >= nstep) break;
                issue_pv(0, q, par, j > 0 ? 1u : 0u);
                if (nt2 == 2) {
                    if (j + 1 < nstep) {
                        if (j > 0) wait(PVDONE + 1, uint32_t(q & 1) ^ 1u);
                        issue_s(1, q + 1, par);
                    }
                    issue_pv(1, q, par, j > 0 ? 1u : 0u);
                }
                if (j + 2 < nstep) {
                    wait(PVDONE, uint32_t(q & 1));
                    issue_s(0, q + 2, par);
                }
            }
        }
        // everything issued has landed before the accumulators are read or given back
        commit(&bar[FIN], el);
        wait_for(&bar[FIN], 0u, failed);
        __syncwarp();
    } else if (t < ntl) {
        // ---- softmax: threads (t, 0, lr) and (t, 1, lr) share a row
        const uint32_t my = tmem + (uint32_t((warp & 3) * 32) << 16);       // this warp's TMEM lanes
        const uint32_t ts = my + t * 128, to = my + 256 + t * 128;
        const int last = !have ? -1 : A.a.causal ? len - n_new + tok : len - 1;
        const int firstk = A.a.window > 0 ? last - A.a.window + 1 : 0;
        const int all_lo = __reduce_max_sync(0xffffffffu, have ? firstk : 0);
        const int all_hi = __reduce_min_sync(0xffffffffu, have ? last : 1 << 30);
        const int nstep = 2 * ntile;
        for (int j = 0; j < nstep; ++j) {
            const uint32_t ph = uint32_t(j) & 1u;
            if (!ready(SFULL + 2 * t + (j & 1), uint32_t(j >> 1) & 1u)) break;
            tc_fence_after();
            const int p0 = base + j * STEP + h * 32;
            const uint32_t th = ts + ph * STEP + h * 32;       // this half's columns: S, then P over the first 16
            uint32_t s[32];
            tmem_ld_32x32b_x32(th, s);
            if (p0 < all_lo || p0 + 31 > all_hi) {             // uniform over the warp
                const int f = firstk - p0, e1 = last - p0;     // columns f .. e1 are seen
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (e < f || e > e1) s[e] = 0xFF800000u;
            }
            float a[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 4)
#pragma unroll
                for (int q = 0; q < 2; ++q) a[q] = max3_nan(a[q], __uint_as_float(s[e + 2 * q]), __uint_as_float(s[e + 2 * q + 1]));
            float mt = max_nan(a[0], a[1]) * cq;
            float* mx = maxes + ((ph * 2 + t) * 2) * 128 + lr;
            mx[h * 128] = mt;
            asm volatile("bar.sync %0, 256;" ::"r"(1 + t) : "memory");
            mt = max_nan(mt, mx[(h ^ 1) * 128]);
            float f = 1.f;
            if (!(mt <= m + LAZY)) {            // also at the first keys and for a NaN
                f = m == -INFINITY ? 0.f : ex2(m - mt);
                l *= f;
                m = mt;
            }
            if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                if (!ready(PVDONE + t, ph ^ 1u)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 16) {
                    uint32_t o[16];
                    tmem_ld_x16(to + c0, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st_x16(to + c0, o);
                }
            }
            const float ref = (m == -INFINITY ? 0.f : m) - UP;
            float2 sum = make_float2(0.f, 0.f), sum2 = sum;
            uint32_t hp[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                            make_float2(cq, cq), make_float2(-ref, -ref));
                const float2 p = make_float2(ex2(x.x), ex2(x.y));
                if (e & 1) sum = __fadd2_rn(sum, p);
                else sum2 = __fadd2_rn(sum2, p);
                hp[e] = pack_h2(p.x, p.y);
            }
            tmem_st_x16(th, hp);
            l += (sum.x + sum.y) + (sum2.x + sum2.y);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[PFULL + 2 * t + (j & 1)]);
        }
        sums[(t * 2 + h) * 128 + lr] = l;
    }
    __syncthreads();
    tc_fence_after();
    if (warp < 16 && t < ntl) {
        const bool bad = *failed != 0;
        l = sums[(t * 2) * 128 + lr] + sums[(t * 2 + 1) * 128 + lr];
        float* part = A.nsplit > 1 ? A.a.ws + (size_t(item) * A.nsplit + split) * (ROWS * (D + 2)) : nullptr;
        E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + tok * A.a.os.t + hq * A.a.os.h;
        const bool vec = (reinterpret_cast<uintptr_t>(op) & 15u) == 0;
        const float il = bad ? __int_as_float(0x7FC00000) : l == 0.f ? 0.f : 1.f / l;
        const uint32_t to = tmem + (uint32_t((warp & 3) * 32) << 16) + 256 + t * 128;
#pragma unroll 1
        for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 32) {
            uint32_t o[32];
            if (ntile > 0) tmem_ld_32x32b_x32(to + c0, o);
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
                    for (int j = 0; j < 8; j += 2)
                        *reinterpret_cast<float2*>(part + size_t(t * 128 + lr) * D + c0 + e + j) =
                            bad ? make_float2(il, il) : make_float2(v[j], v[j + 1]);
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
        if (A.nsplit > 1 && have && h == 0) *reinterpret_cast<float2*>(part + ROWS * D + 2 * (t * 128 + lr)) = make_float2(m, l);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 20) tmem_dealloc(tmem, 512);
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

struct ChunkPlan { int per, nrt, nsplit; int64_t items, tiles; };
ChunkPlan plan_of(const Kv4Attn& a, int sms) {
    ChunkPlan p;
    p.per = a.heads / a.c.heads;
    p.nrt = int((int64_t(a.n_q) * p.per + ROWS - 1) / ROWS);
    p.items = int64_t(p.nrt) * a.c.batch * a.c.heads;
    int64_t keys = a.c.max_ctx;
    if (a.window > 0) keys = std::min<int64_t>(keys, int64_t(a.window) + ROWS / p.per + 1);
    p.tiles = (keys + KEYS - 1) / KEYS + (a.window > 0);
    // stretches of at least two tiles while SMs are left over
    p.nsplit = int(std::max<int64_t>(1, std::min<int64_t>(sms / std::max<int64_t>(p.items, 1), p.tiles / 2)));
    return p;
}

}  // namespace

// 18 us of set-up, 2.2 us per key tile and round of CTAs (1.1 with one row tile), 0.5 us
// per stretch to join; 64 channels take about 0.7 of that.
extern "C" double kie_kv4_chunk_us(const Kv4Attn* a, int sms) {
    const ChunkPlan p = plan_of(*a, sms);
    const bool one = int64_t(a->n_q) * p.per <= 128;
    const double rounds = double((p.items * p.nsplit + sms - 1) / sms), tiles = double((p.tiles + p.nsplit - 1) / p.nsplit);
    return 18.0 + rounds * tiles * (one ? 1.1 : 2.2) * (a->c.dim == 64 ? 0.7 : 1.0) + (p.nsplit > 1 ? (one ? 0.0 : 12.0) + 0.5 * p.nsplit : 0.0);
}

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
