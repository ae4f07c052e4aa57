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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "kie_device.cuh"
#include "kie_kv4.h"

using namespace kie;

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

// Where row `r` of [batch][n][head] rows goes: false when it is not stored.
__device__ __forceinline__ bool place(const Kv4& c, int64_t r, int n, const int32_t* start, const int32_t* n_tok,
                                      int& b, int& t, int& h, int64_t& pos) {
    h = int(r % c.heads);
    const int64_t bt = r / c.heads;
    t = int(bt % n);
    b = int(bt / n);
    if (n_tok && t >= __ldg(n_tok + b)) return false;
    pos = int64_t(__ldg(start + b)) + t;
    return pos >= 0 && pos < c.max_ctx;
}

// ---- store -------------------------------------------------------------------------------------
// A row (one position of one head, K or V) is D/8 lanes with 8 channels each.
template <int T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(Kv4 c, const void* k, const void* v, Kv4Strides ks,
                                                         Kv4Strides vs, int n, const int32_t* start,
                                                         const int32_t* n_tok) {
    using E = typename Elem<T>::type;
    constexpr int LPR = D / 8, BLK = D / 32;
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const int64_t r = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LPR;
    const bool isv = blockIdx.y != 0;
    int b = 0, t = 0, h = 0;
    int64_t pos = 0;
    const bool ok = r < int64_t(c.batch) * n * c.heads && place(c, r, n, start, n_tok, b, t, h, pos);
    const Kv4Strides& s = isv ? vs : ks;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (ok) {
        const E* p = static_cast<const E*>(isv ? v : k) + b * s.b + t * s.t + h * s.h + l * 8;
        load8<T>(p, aligned16(p), x);
    }
    // to fp16, saturating; the format has no NaN: stored as 0
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = x[i] != x[i] ? 0.f : fminf(fmaxf(x[i], -65504.f), 65504.f);
        x[i] = __half2float(__float2half_rn(y));
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
    for (int o = 1; o < c.group / 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
    const float sf = __half2float(sh);
    const float rcp = sf > 0.f ? __frcp_rn(sf) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (x - z) / s by the reciprocal: within 2^-19 of the quotient, so only a
        // value that close to a half needs the division itself
        const float d = x[i] - lo;
        float q = d * rcp;
        const float f = q - floorf(q);
        if (fabsf(f - 0.5f) < 1.f / 65536.f) q = sf > 0.f ? __fdiv_rn(d, sf) : 0.f;
        w |= uint32_t(min(15, int(rintf(q)))) << (4 * i);
    }
    const size_t row = (size_t(b) * c.heads + h) * c.ctx_pad + size_t(pos);
    if (!isv) {
        if (ok) reinterpret_cast<uint32_t*>(c.kc)[row * LPR + (l & 3) * BLK + (l >> 2)] = w;
    } else {
        // lane l stores word l = units (g, 2wi) and (g, 2wi + 1): see kie_kv4.h
        const int g = l / (D / 64), wi = l % (D / 64);
        const int src = (lane - l) + 8 * wi + (g >> 1);
        const uint32_t w0 = __shfl_sync(0xffffffffu, w, src), w1 = __shfl_sync(0xffffffffu, w, src + 4);
        const uint32_t out = __byte_perm(w0, w1, (g & 1) ? 0x7632 : 0x5410);
        if (ok) reinterpret_cast<uint32_t*>(c.vc)[row * LPR + l] = out;
    }
    const int ng = D / c.group, lpg = c.group / 8;
    if (ok && l % lpg == 0) {
        uint16_t* pp = (isv ? c.vp : c.kp) + row * (2 * ng) + l / lpg;
        pp[0] = __half_as_ushort(sh);
        pp[ng] = __half_as_ushort(__float2half_rn(lo));
    }
}

// ---- read back ---------------------------------------------------------------------------------
template <int T, int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4 c, void* k, void* v, Kv4Strides ks, Kv4Strides vs, int n,
                                                       const int32_t* start, const int32_t* n_tok) {
    using E = typename Elem<T>::type;
    constexpr int LPR = D / 8, BLK = D / 32;
    const int l = threadIdx.x % LPR;
    const int64_t r = (int64_t(blockIdx.x) * 256 + threadIdx.x) / LPR;
    const bool isv = blockIdx.y != 0;
    if (r >= int64_t(c.batch) * n * c.heads) return;
    int b, t, h;
    int64_t pos;
    if (!place(c, r, n, start, n_tok, b, t, h, pos)) return;
    const size_t row = (size_t(b) * c.heads + h) * c.ctx_pad + size_t(pos);
    uint32_t w;
    if (!isv) {
        w = reinterpret_cast<const uint32_t*>(c.kc)[row * LPR + (l & 3) * BLK + (l >> 2)];
    } else {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(c.vc) + row * (D / 4) + (2 * (l & 3)) * BLK + (l >> 2);
        w = uint32_t(u[0]) | uint32_t(u[BLK]) << 16;
    }
    const int ng = D / c.group, gi = l * 8 / c.group;
    const uint16_t* pp = (isv ? c.vp : c.kp) + row * (2 * ng);
    const float s = __half2float(__ushort_as_half(pp[gi])), z = __half2float(__ushort_as_half(pp[ng + gi]));
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = fmaf(float((w >> (4 * i)) & 15u), s, z);
        if (T == KV4_F16) f[i] = fminf(fmaxf(f[i], -65504.f), 65504.f);
    }
    const Kv4Strides& st = isv ? vs : ks;
    E* p = static_cast<E*>(isv ? v : k) + b * st.b + t * st.t + h * st.h + l * 8;
    store8<T>(p, aligned16(p), f);
}

// ---- attention ---------------------------------------------------------------------------------
// Work is a list of tiles of TP positions: for every pair (request, tile of RT
// query rows) and K/V head, the tiles that some row of it sees.  The list is cut
// into equal ranges, one per CTA, whatever the requests' lengths; a CTA's range
// meets one or more (pair, head) items and leaves a partial (m, l, o) of each
// that it does not hold whole.  A second kernel joins the partials.
constexpr int TP = 32;        // positions per tile = one warp's step
constexpr int NW = 8;         // warps per CTA, each with its own tiles and copies in flight
constexpr int STG = 3;        // tiles in flight per warp

// HL8: 8 query rows, the operands q and p as fp16 hi + lo in rows r and r + 8
// (22 bits and more: fp32 and fp16 tensors).  S8, S16: 8 or 16 rows, one fp16
// each (bf16 tensors: 11 bits are 8 times finer than their rounding).
enum Mode { HL8 = 0, S8 = 1, S16 = 2 };
__host__ __device__ constexpr int rows_of(int mode) { return mode == S16 ? 16 : 8; }

struct AttnArgs {
    Kv4Attn a;
    int32_t per;             // query heads per K/V head
    int32_t nrt;             // row tiles per request
    int32_t nctas;           // CTAs of the main kernel
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
__device__ __forceinline__ int pair_tiles(const AttnArgs& A, int p, int rt) {
    int lo, hi, len, n;
    pair_keys(A, p / A.nrt, (p % A.nrt) * rt, rt, lo, hi, len, n);
    return hi > lo ? (hi + TP - 1) / TP - lo / TP : 0;
}

// First tile of each CTA's range, of T tiles over n CTAs.
__device__ __forceinline__ int64_t range_begin(int64_t T, int i, int n) { return T * i / n; }

// One warp: total tiles, and the pair that holds tile `at` (with its first tile).
__device__ __forceinline__ int64_t scan_pairs(const AttnArgs& A, int rt, int64_t at_num, int at_den, int& pair,
                                              int64_t& first, int64_t& at) {
    const int lane = threadIdx.x & 31, np = A.a.c.batch * A.nrt;
    int64_t T = 0;
    for (int p0 = 0; p0 < np; p0 += 32) T += p0 + lane < np ? pair_tiles(A, p0 + lane, rt) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
    T *= A.a.c.heads;
    at = T * at_num / at_den;
    pair = np;
    first = T;
    int64_t run = 0;
    for (int p0 = 0; p0 < np; p0 += 32) {
        const int64_t own = p0 + lane < np ? int64_t(pair_tiles(A, p0 + lane, rt)) * A.a.c.heads : 0;
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

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127
// Four codes pairs of a word whose halves hold two elements' nibbles: element
// values code * 2^-24 * {1, 16, 1, 16}.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t* r) {
    r[0] = w & 0x000F000Fu;
    r[1] = w & 0x00F000F0u;
    r[2] = (w >> 8) & 0x000F000Fu;
    r[3] = (w >> 8) & 0x00F000F0u;
}
// 16-byte copy global -> shared of the first n (0..16) bytes, zeros after them.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <int D, int NG>
struct Tile {
    static constexpr int CODES = TP * D / 2, PAR = TP * 4 * NG, BYTES = 2 * (CODES + PAR);
};

// The NG scales (or zeros) of a position, as floats.
template <int NG>
__device__ __forceinline__ void scales(const uint8_t* par, int pos, float* s) {
    if (NG == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(par + pos * 16);
        const float2 a = h2_to_f2(w.x), b = h2_to_f2(w.y);
        s[0] = a.x; s[1] = a.y; s[2 % NG] = b.x; s[3 % NG] = b.y;
    } else if (NG == 2) {
        const float2 a = h2_to_f2(*reinterpret_cast<const uint32_t*>(par + pos * 8));
        s[0] = a.x; s[1 % NG] = a.y;
    } else {
        s[0] = h2_to_f2(*reinterpret_cast<const uint32_t*>(par + pos * 4)).x;
    }
}

template <int D, int NG, int MODE, int T>
__global__ void __launch_bounds__(NW * 32, 1) kv4_attention_kernel(const AttnArgs A) {
    using E = typename Elem<T>::type;
    using TL = Tile<D, NG>;
    constexpr int RT = rows_of(MODE), BLK = D / 32, BPG = BLK / NG;   // 32-channel blocks, per group
    constexpr int RPL = MODE == S16 ? 2 : 1;                          // query rows per lane
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_plan[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * (STG * TL::BYTES);
    const uint32_t ring_u = smem_u32(ring);
    const Kv4& c = A.a.c;

    if (warp == 0) {
        int pair;
        int64_t first, at;
        const int64_t total = scan_pairs(A, RT, blockIdx.x, A.nctas, pair, first, at);
        const int64_t end = range_begin(total, blockIdx.x + 1, A.nctas);
        if (lane == 0) { s_plan[0] = at; s_plan[1] = end; s_plan[2] = pair; s_plan[3] = first; }
    }
    __syncthreads();
    // let the joining kernel's blocks come up: they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int64_t at = s_plan[0];
    const int64_t end = s_plan[1];
    int pair = int(s_plan[2]);
    int64_t first = s_plan[3];       // first tile of the pair
    while (at < end) {
        const int nt = pair_tiles(A, pair, RT);
        if (at >= first + int64_t(nt) * c.heads) { first += int64_t(nt) * c.heads; ++pair; continue; }
        const int head = int((at - first) / nt);
        const int tile0 = int((at - first) % nt);
        const int ntile = int(min(int64_t(nt - tile0), end - at));
        at += ntile;
        const int b = pair / A.nrt, r0 = (pair % A.nrt) * RT;
        int lo, hi, len, n_new;
        pair_keys(A, b, r0, RT, lo, hi, len, n_new);
        const int base = lo / TP * TP + tile0 * TP;           // first position of this segment
        const size_t row0 = (size_t(b) * c.heads + head) * c.ctx_pad;
        const uint8_t* src[4] = {c.kc + row0 * (D / 2), c.vc + row0 * (D / 2),
                                 reinterpret_cast<const uint8_t*>(c.kp) + row0 * (4 * NG),
                                 reinterpret_cast<const uint8_t*>(c.vp) + row0 * (4 * NG)};
        // copies of tile i of the segment into ring stage st; positions from len on become zeros
        auto copy_tile = [&](int i, int st) {
            const int p0 = base + i * TP, nv = min(TP, len - p0);   // valid positions (> 0)
            const uint32_t dst = ring_u + st * TL::BYTES;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const uint8_t* gsrc = src[a] + size_t(p0) * (D / 2);
                const int nb = nv * (D / 2);
#pragma unroll
                for (int j = 0; j < TL::CODES / 512; ++j) {
                    const int o = (j * 32 + lane) * 16;
                    copy16(dst + a * TL::CODES + o, gsrc + o, o < nb ? 16 : 0);
                }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const uint8_t* gsrc = src[2 + a] + size_t(p0) * (4 * NG);
                const int nb = nv * (4 * NG);
#pragma unroll
                for (int j = 0; j < (TL::PAR + 511) / 512; ++j) {
                    const int o = (j * 32 + lane) * 16;
                    if (o < TL::PAR)
                        copy16(dst + 2 * TL::CODES + a * TL::PAR + o, gsrc + o, min(16, max(0, nb - o)));
                }
            }
        };
#pragma unroll
        for (int s = 0; s < STG - 1; ++s) {
            if (warp + s * NW < ntile) copy_tile(warp + s * NW, s);
            cp_async_commit();
        }

        // ---- this lane's query rows as operands
        uint32_t qa[BLK][2][4];        // [block][mma][a0..a3]
        uint32_t qz[2];                // sums of q over the groups: a0, a1 of the zeros' mma
        float cq[RPL];                 // from the mma's units to log2 units of the softmax
        int last[RPL], firstk[RPL];    // keys the row sees: firstk .. last
        int all_lo = 0, all_hi = 1 << 30;   // positions that every row of the tile sees
#pragma unroll
        for (int rr = 0; rr < RPL; ++rr) {
            const int r = r0 + g + rr * 8;
            const bool have = r < n_new * A.per;
            const int tok = have ? r / A.per : 0, hq = head * A.per + (have ? r % A.per : 0);
            last[rr] = !have ? -1 : A.a.causal ? len - n_new + tok : len - 1;
            firstk[rr] = A.a.window > 0 && A.a.causal ? last[rr] - A.a.window + 1 : 0;
            if (have) { all_lo = max(all_lo, firstk[rr]); all_hi = min(all_hi, last[rr]); }
            const E* qp = static_cast<const E*>(A.a.q) + b * A.a.qs.b + tok * A.a.qs.t + hq * A.a.qs.h;
            float x[BLK][8], mx = 0.f, sum[NG];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) sum[gi] = 0.f;
#pragma unroll
            for (int i = 0; i < BLK; ++i) {
                const E* p = qp + i * 32 + t * 8;
                if (have) load8<T>(p, aligned16(p), x[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!have) x[i][j] = 0.f;
                    mx = fmaxf(mx, fabsf(x[i][j]));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // exact power of two that brings the row's largest element to [2^11, 2^12)
            int e = ((__float_as_int(mx) >> 23) & 255) - 127;
            e = min(max(e, -100), 114);
            const float up = pow2i(11 - e);
            cq[rr] = A.a.scale * 1.4426950408889634f * pow2i(e - 11 + 24);
#pragma unroll
            for (int i = 0; i < BLK; ++i) {
                float hi_[8], lo_[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = x[i][j] * up;
                    sum[i / BPG] += y;
                    hi_[j] = __half2float(__float2half_rn(y));
                    lo_[j] = y - hi_[j];
                    const float f = (j & 1) ? 1.f / 16.f : 1.f;
                    hi_[j] *= f;
                    lo_[j] *= f;
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int j = 2 * m + s;
                        const uint32_t h2 = pack_h2(hi_[j], hi_[j + 4]);
                        if (MODE == S16) qa[i][m][2 * s + rr] = h2;
                        else {
                            qa[i][m][2 * s] = h2;
                            qa[i][m][2 * s + 1] = MODE == HL8 ? pack_h2(lo_[j], lo_[j + 4]) : 0u;
                        }
                    }
            }
            // zeros' operand: k = 2t', 2t'+1 are a pair of groups, hi for t' < 2, lo after
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 1);
                sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 2);
                sum[gi] *= 1.f / 256.f;
            }
            float s0 = 0.f, s1 = 0.f;
            if (NG == 4) { s0 = (t & 1) ? sum[2 % NG] : sum[0]; s1 = (t & 1) ? sum[3 % NG] : sum[1 % NG]; }
            if (NG == 2 && (t & 1) == 0) { s0 = sum[0]; s1 = sum[1 % NG]; }
            if (NG == 1 && (t & 1) == 0) s1 = sum[0];     // the pair is (scale, zero)
            const float h0 = __half2float(__float2half_rn(s0)), h1 = __half2float(__float2half_rn(s1));
            const uint32_t zz = t < 2 ? pack_h2(h0, h1) : pack_h2(s0 - h0, s1 - h1);
            qz[rr] = zz;
            if (RPL == 1) qz[1] = 0u;
        }
        const int zoff = NG == 4 ? 8 + (t & 1) * 4 : NG == 2 ? 4 : 0;

        float o[BLK][4][4];            // [block][nibble][c0..c3]
        float zl[4] = {0.f, 0.f, 0.f, 0.f};
        float m[RPL];
        int ev = 1;                    // biased fp16 exponent of the largest V scale so far
#pragma unroll
        for (int i = 0; i < BLK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][j][k] = 0.f;
#pragma unroll
        for (int rr = 0; rr < RPL; ++rr) m[rr] = -INFINITY;
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);

        int st = 0;
        for (int i = warp; i < ntile; i += NW) {
            {
                const int nx = i + (STG - 1) * NW;
                int ns = st + STG - 1;
                if (ns >= STG) ns -= STG;
                __syncwarp();          // every lane is done with the stage that this overwrites
                if (nx < ntile) copy_tile(nx, ns);
                cp_async_commit();
            }
            cp_async_wait_group<STG - 1>();
            __syncwarp();
            const uint8_t* kc = ring + st * TL::BYTES;
            const uint8_t* vc = kc + TL::CODES;
            const uint8_t* kp = vc + TL::CODES;
            const uint8_t* vp = kp + TL::PAR;
            if (++st == STG) st = 0;
            const int p0 = base + i * TP;

            // ---- scores of 32 positions: x[tile][row][2]
            float x[4][RPL][2];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int pos = n * 8 + g;
                uint32_t w[BLK];
                if (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(kc + pos * 64 + t * 16);
                    w[0] = v.x; w[1] = v.y; w[2 % BLK] = v.z; w[3 % BLK] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(kc + pos * 32 + t * 8);
                    w[0] = v.x; w[1] = v.y;
                }
                float z[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t az[4] = {qz[0], qz[1], 0u, 0u};
                mma16816(z, az, *reinterpret_cast<const uint32_t*>(kp + pos * 4 * NG + zoff), 0u);
                float s0[NG], s1[NG];
                scales<NG>(kp, n * 8 + 2 * t, s0);
                scales<NG>(kp, n * 8 + 2 * t + 1, s1);
                float y[RPL][2];
#pragma unroll
                for (int rr = 0; rr < RPL; ++rr) {
                    y[rr][0] = z[2 * rr] * (1.f / 65536.f);
                    y[rr][1] = z[2 * rr + 1] * (1.f / 65536.f);
                }
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < BPG; ++j) {
                        uint32_t r[4];
                        unpack4(w[gi * BPG + j], r);
                        mma16816(acc, qa[gi * BPG + j][0], r[0], r[1]);
                        mma16816(acc, qa[gi * BPG + j][1], r[2], r[3]);
                    }
                    if (MODE == HL8) { acc[0] += acc[2]; acc[1] += acc[3]; }
#pragma unroll
                    for (int rr = 0; rr < RPL; ++rr) {
                        y[rr][0] = fmaf(acc[2 * rr], s0[gi], y[rr][0]);
                        y[rr][1] = fmaf(acc[2 * rr + 1], s1[gi], y[rr][1]);
                    }
                }
#pragma unroll
                for (int rr = 0; rr < RPL; ++rr) {
                    x[n][rr][0] = y[rr][0] * cq[rr];
                    x[n][rr][1] = y[rr][1] * cq[rr];
                }
            }
            if (p0 < all_lo || p0 + TP - 1 > all_hi) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int rr = 0; rr < RPL; ++rr)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int p = p0 + n * 8 + 2 * t + k;
                            if (p < firstk[rr] || p > last[rr]) x[n][rr][k] = -INFINITY;
                        }
            }
            // ---- running maximum, and the largest V scale of the tile
            float corr[RPL], mref[RPL];
            bool grew = false;
#pragma unroll
            for (int rr = 0; rr < RPL; ++rr) {
                float mx = x[0][rr][0];
#pragma unroll
                for (int n = 0; n < 4; ++n) mx = max_nan(mx, max_nan(x[n][rr][0], x[n][rr][1]));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = max_nan(m[rr], mx);
                grew |= mn > m[rr];
                mref[rr] = (mn == -INFINITY ? 0.f : mn) - 15.f;      // p <= 2^15: fp16's range, used whole
                corr[rr] = ex2(m[rr] - 15.f - mref[rr]);
                m[rr] = mn;
            }
            uint32_t sb;
            if (NG == 4) {
                const uint2 w = *reinterpret_cast<const uint2*>(vp + lane * 16);
                const uint32_t a = __vmaxu2(w.x, w.y);
                sb = max(a & 0xFFFFu, a >> 16);
            } else if (NG == 2) {
                const uint32_t a = *reinterpret_cast<const uint32_t*>(vp + lane * 8);
                sb = max(a & 0xFFFFu, a >> 16);
            } else {
                sb = *reinterpret_cast<const uint32_t*>(vp + lane * 4) & 0xFFFFu;
            }
            const int en = max(ev, int(__reduce_max_sync(0xffffffffu, sb) >> 10));
            if (__any_sync(0xffffffffu, grew) || en > ev) {
                const float fe = pow2i(ev - en);
                ev = en;
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    const float cz = corr[RPL == 2 ? rr : 0], co = cz * fe;
                    zl[2 * rr] *= cz;
                    zl[2 * rr + 1] *= cz;
#pragma unroll
                    for (int i2 = 0; i2 < BLK; ++i2)
#pragma unroll
                        for (int j = 0; j < 4; ++j) { o[i2][j][2 * rr] *= co; o[i2][j][2 * rr + 1] *= co; }
                }
            }
            const float fv = pow2i(14 - ev);    // 2^-(E+1), E = ev - 15: p * s * fv < 2^15
            // ---- o += p v, 16 positions at a time
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int pp[4] = {hh * 16 + 2 * t, hh * 16 + 2 * t + 1, hh * 16 + 8 + 2 * t, hh * 16 + 9 + 2 * t};
                float p[RPL][4];
#pragma unroll
                for (int rr = 0; rr < RPL; ++rr)
#pragma unroll
                    for (int k = 0; k < 4; ++k) p[rr][k] = ex2(x[2 * hh + (k >> 1)][rr][k & 1] - mref[rr]);
                // zeros and the row sum: columns 0..NG-1 are the groups' zeros, column NG is 1
                {
                    uint32_t a[4];
                    if (MODE == S16) {
#pragma unroll
                        for (int rr = 0; rr < RPL; ++rr) { a[rr] = pack_h2(p[rr][0], p[rr][1]); a[2 + rr] = pack_h2(p[rr][2], p[rr][3]); }
                    } else {
                        a[0] = pack_h2(p[0][0], p[0][1]);
                        a[2] = pack_h2(p[0][2], p[0][3]);
                        a[1] = a[3] = 0u;
                        if (MODE == HL8) {
                            const float2 h0 = h2_to_f2(a[0]), h1 = h2_to_f2(a[2]);
                            a[1] = pack_h2(p[0][0] - h0.x, p[0][1] - h0.y);
                            a[3] = pack_h2(p[0][2] - h1.x, p[0][3] - h1.y);
                        }
                    }
                    uint32_t b0 = g == NG ? 0x3C003C00u : 0u, b1 = b0;
                    if (g < NG) {
                        const uint8_t* zp = vp + 2 * NG + 2 * g;
                        auto zh = [&](int q) { return uint32_t(*reinterpret_cast<const uint16_t*>(zp + pp[q] * 4 * NG)); };
                        b0 = zh(0) | zh(1) << 16;
                        b1 = zh(2) | zh(3) << 16;
                    }
                    mma16816(zl, a, b0, b1);
                }
                float sv[4][NG];
#pragma unroll
                for (int k = 0; k < 4; ++k) scales<NG>(vp, pp[k], sv[k]);
#pragma unroll
                for (int rr = 0; rr < RPL; ++rr)
#pragma unroll
                    for (int k = 0; k < 4; ++k) p[rr][k] *= fv;
                uint32_t vw[4][D / 64];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (D == 128) {
                        const uint2 v = *reinterpret_cast<const uint2*>(vc + pp[k] * 64 + g * 8);
                        vw[k][0] = v.x; vw[k][1 % (D / 64)] = v.y;
                    } else {
                        vw[k][0] = *reinterpret_cast<const uint32_t*>(vc + pp[k] * 32 + g * 4);
                    }
                }
                uint32_t a[4];
#pragma unroll
                for (int i2 = 0; i2 < BLK; ++i2) {
                    if (i2 % BPG == 0) {     // p * s of the group
                        const int gi = i2 / BPG;
#pragma unroll
                        for (int rr = 0; rr < RPL; ++rr) {
                            const float y0 = p[rr][0] * sv[0][gi], y1 = p[rr][1] * sv[1][gi];
                            const float y2 = p[rr][2] * sv[2][gi], y3 = p[rr][3] * sv[3][gi];
                            if (MODE == S16) {
                                a[rr] = pack_h2(y0, y1);
                                a[2 + rr] = pack_h2(y2, y3);
                            } else {
                                a[0] = pack_h2(y0, y1);
                                a[2] = pack_h2(y2, y3);
                                a[1] = a[3] = 0u;
                                if (MODE == HL8) {
                                    const float2 h0 = h2_to_f2(a[0]), h1 = h2_to_f2(a[2]);
                                    a[1] = pack_h2(y0 - h0.x, y1 - h0.y);
                                    a[3] = pack_h2(y2 - h1.x, y3 - h1.y);
                                }
                            }
                        }
                    }
                    const int wi = i2 >> 1;
                    const uint32_t sel = (i2 & 1) ? 0x7632u : 0x5410u;
                    uint32_t r0_[4], r1_[4];
                    unpack4(__byte_perm(vw[0][wi], vw[1][wi], sel), r0_);
                    unpack4(__byte_perm(vw[2][wi], vw[3][wi], sel), r1_);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16816(o[i2][j], a, r0_[j], r1_[j]);
                }
            }
        }
        cp_async_wait_group<0>();
        __syncthreads();               // every warp is done with its ring: it becomes the merge buffer

        // ---- merge the warps: [warp][RT][D] sums, [warp][RT][8] zeros and row sums, [warp][RT] maxima
        float* mo = reinterpret_cast<float*>(smem);
        float* mz = mo + NW * RT * D;
        float* mm = mz + NW * RT * 8;
        const float back = pow2i(ev - 14) * 16777216.f;   // undo fv and the codes' 2^-24
#pragma unroll
        for (int rr = 0; rr < RPL; ++rr) {
            const int row = warp * RT + g + rr * 8;
#pragma unroll
            for (int i = 0; i < BLK; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4 v;
                    float* e = &v.x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y = MODE == HL8 ? o[i][j][k] + o[i][j][2 + k] : o[i][j][2 * rr + k];
                        e[j] = y * (back * ((j & 1) ? 1.f / 16.f : 1.f));
                    }
                    *reinterpret_cast<float4*>(mo + size_t(row) * D + i * 32 + t * 8 + k * 4) = v;
                }
            mz[row * 8 + 2 * t] = MODE == HL8 ? zl[0] + zl[2] : zl[2 * rr];
            mz[row * 8 + 2 * t + 1] = MODE == HL8 ? zl[1] + zl[3] : zl[2 * rr + 1];
            if (t == 0) mm[row] = m[rr];
        }
        __syncthreads();
        const bool whole = ntile == nt;
        float* part = A.a.ws + (size_t(pair) * c.heads + head + blockIdx.x) * (RT * (D + 2));
        for (int i = threadIdx.x; i < RT * D; i += NW * 32) {
            const int r = i / D, d = i % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = max_nan(M, mm[w * RT + r]);
            float os = 0.f, ls = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float mw = mm[w * RT + r];
                const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
                os = fmaf(f, mo[(w * RT + r) * D + d] + mz[(w * RT + r) * 8 + d / (D / NG)], os);
                ls = fmaf(f, mz[(w * RT + r) * 8 + NG], ls);
            }
            if (whole) {
                const int row = r0 + r;
                if (row < n_new * A.per) {
                    E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + (row / A.per) * A.a.os.t +
                            (head * A.per + row % A.per) * A.a.os.h;
                    op[d] = Elem<T>::from(ls == 0.f ? 0.f : os / ls);
                }
            } else {
                part[i] = os;
                if (d == 0) { part[RT * D + 2 * r] = M; part[RT * D + 2 * r + 1] = ls; }
            }
        }
        __syncthreads();               // the merge buffer becomes the ring again
    }
}

// Join the partials of every item that more than one CTA worked on; items
// without a key get zeros.  One block per (pair, K/V head).
template <int D, int RT, int T>
__global__ void __launch_bounds__(256) kv4_join_kernel(const AttnArgs A) {
    using E = typename Elem<T>::type;
    __shared__ int64_t s_at[3];
    const int pair = blockIdx.x / A.a.c.heads, head = blockIdx.x % A.a.c.heads;
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
    // every block waits for the main kernel, also one with nothing to join: what
    // follows in the stream waits for this kernel alone
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t total = s_at[1];
    int lo, hi, len, n_new;
    const int b = pair / A.nrt, r0 = (pair % A.nrt) * RT;
    pair_keys(A, b, r0, RT, lo, hi, len, n_new);
    const int rows = min(RT, n_new * A.per - r0);
    if (rows <= 0) return;
    const int nt = pair_tiles(A, pair, RT);
    const int64_t t0 = s_at[0] + int64_t(head) * nt, t1 = t0 + nt;
    int c0 = 0, c1 = 0;                 // CTAs c0 .. c1 hold tiles of this item
    if (nt > 0) {
        // CTA of tile x: the largest i with total * i / n <= x
        auto owner = [&](int64_t x) {
            int64_t i = (x * A.nctas) / total;
            while (i + 1 < A.nctas && range_begin(total, int(i + 1), A.nctas) <= x) ++i;
            while (i > 0 && range_begin(total, int(i), A.nctas) > x) --i;
            return int(i);
        };
        c0 = owner(t0);
        c1 = owner(t1 - 1);
        if (c0 == c1) return;           // one CTA held it whole and wrote the result
    }
    const float* part = A.a.ws + (size_t(pair) * A.a.c.heads + head) * (RT * (D + 2));
    for (int i = threadIdx.x; i < rows * D; i += 256) {
        const int r = i / D, d = i % D;
        float M = -INFINITY, ls = 0.f, os = 0.f;
        if (nt > 0)
            for (int k = c0; k <= c1; ++k) {
                if (range_begin(total, k, A.nctas) == range_begin(total, k + 1, A.nctas)) continue;   // an empty range
                const float* pk = part + size_t(k) * (RT * (D + 2));
                const float mk = __ldcg(pk + RT * D + 2 * r);
                if (mk == -INFINITY) continue;
                const float mn = max_nan(M, mk), f0 = ex2(M - mn), f1 = ex2(mk - mn);
                ls = ls * f0 + __ldcg(pk + RT * D + 2 * r + 1) * f1;
                os = os * f0 + __ldcg(pk + i) * f1;
                M = mn;
            }
        const int row = r0 + r;
        E* op = static_cast<E*>(A.a.out) + b * A.a.os.b + (row / A.per) * A.a.os.t + (head * A.per + row % A.per) * A.a.os.h;
        op[d] = Elem<T>::from(ls == 0.f ? 0.f : os / ls);
    }
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

template <int D, int NG, int MODE, int T>
cudaError_t launch_attention(const AttnArgs& A, cudaStream_t st) {
    constexpr int RT = rows_of(MODE);
    constexpr int ring = NW * STG * Tile<D, NG>::BYTES, merge = NW * RT * (D + 9) * 4;
    constexpr int smem = ring > merge ? ring : merge;
    static std::atomic<uint64_t> done{0};
    cudaError_t r = opt_in(kv4_attention_kernel<D, NG, MODE, T>, smem, done);
    if (r != cudaSuccess) return r;
    kv4_attention_kernel<D, NG, MODE, T><<<A.nctas, NW * 32, smem, st>>>(A);
    r = cudaGetLastError();
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(A.a.c.batch) * A.nrt * A.a.c.heads);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, RT, T>, A);
}

template <int D, int NG>
cudaError_t launch_attention_t(const AttnArgs& A, int mode, cudaStream_t st) {
    if (A.a.type == KV4_F16) return launch_attention<D, NG, HL8, KV4_F16>(A, st);
    if (A.a.type == KV4_F32) return launch_attention<D, NG, HL8, KV4_F32>(A, st);
    return mode == S8 ? launch_attention<D, NG, S8, KV4_BF16>(A, st) : launch_attention<D, NG, S16, KV4_BF16>(A, st);
}

template <int T>
cudaError_t append_t(const Kv4& c, const void* k, const void* v, const Kv4Strides& ks, const Kv4Strides& vs, int n,
                     const int32_t* start, const int32_t* n_tok, cudaStream_t st) {
    const int64_t threads = int64_t(c.batch) * n * c.heads * (c.dim / 8);
    const dim3 grid(unsigned((threads + 255) / 256), 2);
    if (c.dim == 128) kv4_append_kernel<T, 128><<<grid, 256, 0, st>>>(c, k, v, ks, vs, n, start, n_tok);
    else kv4_append_kernel<T, 64><<<grid, 256, 0, st>>>(c, k, v, ks, vs, n, start, n_tok);
    return cudaGetLastError();
}
template <int T>
cudaError_t read_t(const Kv4& c, void* k, void* v, const Kv4Strides& ks, const Kv4Strides& vs, int n,
                   const int32_t* start, const int32_t* n_tok, cudaStream_t st) {
    const int64_t threads = int64_t(c.batch) * n * c.heads * (c.dim / 8);
    const dim3 grid(unsigned((threads + 255) / 256), 2);
    if (c.dim == 128) kv4_read_kernel<T, 128><<<grid, 256, 0, st>>>(c, k, v, ks, vs, n, start, n_tok);
    else kv4_read_kernel<T, 64><<<grid, 256, 0, st>>>(c, k, v, ks, vs, n, start, n_tok);
    return cudaGetLastError();
}

}  // namespace

extern "C" cudaError_t kie_launch_kv4_append(const Kv4* c, const void* k, const void* v, const Kv4Strides* ks,
                                             const Kv4Strides* vs, int type, int n, const int32_t* start,
                                             const int32_t* n_tok, cudaStream_t st) {
    if (type == KV4_F16) return append_t<KV4_F16>(*c, k, v, *ks, *vs, n, start, n_tok, st);
    if (type == KV4_BF16) return append_t<KV4_BF16>(*c, k, v, *ks, *vs, n, start, n_tok, st);
    return append_t<KV4_F32>(*c, k, v, *ks, *vs, n, start, n_tok, st);
}

extern "C" cudaError_t kie_launch_kv4_read(const Kv4* c, void* k, void* v, const Kv4Strides* ks, const Kv4Strides* vs,
                                           int type, int n, const int32_t* start, const int32_t* n_tok,
                                           cudaStream_t st) {
    if (type == KV4_F16) return read_t<KV4_F16>(*c, k, v, *ks, *vs, n, start, n_tok, st);
    if (type == KV4_BF16) return read_t<KV4_BF16>(*c, k, v, *ks, *vs, n, start, n_tok, st);
    return read_t<KV4_F32>(*c, k, v, *ks, *vs, n, start, n_tok, st);
}

// A partial of CTA i for item k lies at slot k + i: a CTA's items and an item's
// CTAs are both consecutive, so no two (item, CTA) pairs that meet share a slot.
extern "C" size_t kie_kv4_attention_ws_floats(const Kv4* c, int heads, int n_q, int type, int sms) {
    const int64_t rows = int64_t(n_q) * (heads / c->heads);
    const int rt = rows_of(mode_of(type, rows > 8 ? 16 : 8));
    const size_t items = size_t(c->batch) * size_t((rows + rt - 1) / rt) * c->heads;
    return (items + size_t(sms)) * rt * (c->dim + 2);
}

extern "C" cudaError_t kie_launch_kv4_attention(const Kv4Attn* a, int sms, cudaStream_t st) {
    AttnArgs A;
    A.a = *a;
    A.per = a->heads / a->c.heads;
    const int64_t rows = int64_t(a->n_q) * A.per;
    const int mode = mode_of(a->type, rows > 8 ? 16 : 8);
    A.nrt = int((rows + rows_of(mode) - 1) / rows_of(mode));
    A.nctas = sms;
    const int ng = a->c.dim / a->c.group;
    if (a->c.dim == 128) {
        if (ng == 4) return launch_attention_t<128, 4>(A, mode, st);
        if (ng == 2) return launch_attention_t<128, 2>(A, mode, st);
        return launch_attention_t<128, 1>(A, mode, st);
    }
    if (ng == 2) return launch_attention_t<64, 2>(A, mode, st);
    return launch_attention_t<64, 1>(A, mode, st);
}
