// A token per row of logits by temperature, top-k, top-p and min-p from given
// random numbers.
//
// With m the row's largest logit and w_i = exp((l_i - m) / T), the tokens kept
// are a prefix of the order (logit descending, index ascending), cut by top-k
// (length), top-p (the shortest prefix with p of the top-k prefix's mass) and
// min-p (w_i >= min_p); the drawn token is the first, in index order, at which
// the running mass of the kept tokens passes u times their total.
//
// Tokens are whole numbers, so the masses that decide them must not depend on
// the order of a sum: w_i is computed to about 2^-43 in pairs of fp32 numbers
// (fp64 runs at 1/64 of their rate here) and kept as an integer count of
// 2^-44.  Sums of integers are exact in any order, so the threads, the shared-
// memory atomics and the CTAs of a cluster give one answer, and a token differs
// from the definition's only where u falls within about 2^-37 of a border.
//
// One cluster per row, the row's logits read once into its CTAs' shared memory.
// y = (m - l) log2(e) / T puts the logits into bins of 1/16.  No sort of the row:
//   a small top-k: the counts of the bins say which hold the first k; their few
//     tokens go to one CTA, which sorts them and applies every filter there;
//   top-p alone: masses to 2^-15 in bins of 1/64 say between which bins the prefix
//     must end; one pass of exact weights sums what lies before and after, and lists
//     those bins' tokens, which one CTA sorts;
//   otherwise (a top-k above 512, or more than 1,024 tokens in those bins): histograms
//     of exact masses, then over the bits of the logit, a thousand steps each, until
//     one value or a few tokens are left.
//
// The bytes would take 0.02 us for a row of 32,000 and 4.9 us for 64 of 131,072; what
// bounds it is, for few rows, the chain of passes and of cluster barriers, and for many
// the 45 instructions of an exact weight.
// Measured (us; unfiltered / top-k 50 / top-p 0.9): 1 x 32,000 fp32 8.2 / 13.1 / 20.1 (greedy
// 5.2); 8 x 50,001 bf16 9.6 / 14.1 / 23.7; 64 x 32,000 fp32 13 / 15 / 29; 256 x 32,000 35 / 34
// / 71; 64 x 131,072 38 / 41 / 84 (greedy 17: what reading and the first barrier take).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "kie_device.cuh"
#include "kie_sample.h"

namespace cg = cooperative_groups;

namespace {

constexpr int NT = 512, NWARP = NT / 32;   // threads per CTA
constexpr int NB = 1024;                   // histogram bins (two per thread)
constexpr int NF = 4 * NB;                 // bins of the approximate masses, a quarter as wide
constexpr int FRAC = 44;                   // masses count 2^-44
constexpr int LIST = 32;                   // candidates resolved by one warp
constexpr int MAXC = 8;                    // CTAs per row
// The sorted paths: largest top-k, most candidates.  Top-k 400 of 32,000: 15.6 us sorted, and
// 2,000 22 by histograms.
constexpr int KLIM = 512, CAP = 1024;

// 2^(-j/128) * 2^60, by the series of exp(-j ln 2 / 128) (to 2^-52)
struct Pow2 { uint64_t v[128]; };
constexpr Pow2 make_pow2() {
    Pow2 t{};
    for (int j = 0; j < 128; ++j) {
        const double a = -0.693147180559945309417 * j / 128.0;
        double s = 0.0;
        for (int k = 24; k >= 1; --k) s = (1.0 + s) * a / k;   // a + a^2/2! + ...
        t.v[j] = uint64_t((1.0 + s) * 1152921504606846976.0);
    }
    return t;
}
__device__ constexpr Pow2 kPow2 = make_pow2();

struct Shared {
    uint32_t h[4][NB];          // local histogram: counts, three 15-bit limbs of the masses
    uint32_t fc[2][NB];         // this CTA's share of the summed histogram: counts, masses
    uint64_t fm[2][NB];         // sorted paths: masses, sort keys
    uint64_t table[128];        // 2^(-j/128) * 2^60
    uint64_t xch[4][4];         // values other CTAs read, by exchange number
    uint64_t list_w[LIST];
    uint32_t list_key[LIST];
    int32_t list_idx[LIST];
    uint32_t list_n;
    uint64_t wsum[NWARP];
    uint32_t wcnt[NWARP];
    uint32_t wmin[NWARP], wmax[NWARP];
    // result of find()
    int32_t f_bin;
    uint32_t f_cnt, f_n;
    uint64_t f_mass;
    // result of select()
    uint32_t key, n_eq, all_eq, last;
    uint64_t mass;
    float chi, clo;
};

template <int T> __device__ __forceinline__ float to_float(const void* p, int64_t i);
template <> __device__ __forceinline__ float to_float<0>(const void* p, int64_t i) { return __half2float(static_cast<const __half*>(p)[i]); }
template <> __device__ __forceinline__ float to_float<1>(const void* p, int64_t i) { return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]); }
template <> __device__ __forceinline__ float to_float<2>(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }

// Order-preserving integer of a logit (-0 and 0 are one value): of its own 16 bits
// where the type has no more, so that neighbours differ by one.
template <int T>
__device__ __forceinline__ uint32_t key_of(float x) {
    if (T == 0) {
        const uint32_t b = __half_as_ushort(__float2half_rn(x + 0.f));
        return b & 0x8000u ? 0xFFFFu & ~b : b | 0x8000u;
    }
    const uint32_t b = __float_as_uint(x + 0.f), k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return T == 1 ? k >> 16 : k;
}
template <int T>
__device__ __forceinline__ float of_key(uint32_t k) {
    if (T == 0) return __half2float(__ushort_as_half(uint16_t(k & 0x8000u ? k & 0x7FFFu : ~k)));
    if (T == 1) return __uint_as_float((k & 0x8000u ? k & 0x7FFFu : 0xFFFFu & ~k) << 16);
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// What weights need of a row: its maximum and log2(e)/T as a sum of two floats.
struct Row {
    float m, chi, clo;
    const uint64_t* table;
    // (m - l) log2(e) / T in fp32: monotone in l
    __device__ __forceinline__ float y(float l) const { return (m - l) * chi; }
    // exp((l - m) / T) in units of 2^-44, to about 2^-39 relative.  Floats become
    // integers by adding 1.5 * 2^23 and reading the bits: conversions run at an
    // eighth of the additions' rate.
    __device__ __forceinline__ uint64_t weight(float l) const {
        constexpr float MAGIC = 12582912.f;
        constexpr int MAGIC_BITS = 0x4B400000;
        const float hi = m - l;
        const float bb = hi - m, lo = (m - (hi - bb)) - (l + bb);   // m - l = hi + lo exactly
        const float yh = hi * chi;
        const float yl = fmaf(hi, clo, fmaf(lo, chi, fmaf(hi, chi, -yh)));
        // y = k / 128 + f + yl, |f| <= 1/256, f exact
        const float kr = fmaf(yh, 128.f, MAGIC);
        const float f = fmaf(kr - MAGIC, -1.f / 128.f, yh);
        const int k = __float_as_int(kr) - MAGIC_BITS;
        // 2^-(f + yl) = 1 - a + a^2/2 - ..., a = (f + yl) ln 2 = ah + al
        constexpr float L1 = 0.693147182464599609375f, L2 = -1.904654299957767e-9f;   // ln 2 = L1 + L2
        const float ah = f * L1;
        const float al = fmaf(yl, L1, fmaf(f, L2, fmaf(f, L1, -ah)));
        const float q = fmaf(ah * ah, fmaf(ah, fmaf(ah, 1.f / 24.f, -1.f / 6.f), 0.5f), al * fmaf(al, 0.5f, fmaf(ah * ah, -0.5f, ah)));
        // that minus 1 in units of 2^-39: a's large part in two exact steps, the rest (below 2^-17) in one
        const float r1 = fmaf(ah, 1048576.f, MAGIC);                              // 2^20
        const float r2 = fmaf(fmaf(ah, 1048576.f, -(r1 - MAGIC)), 524288.f, MAGIC);   // 2^19 more
        const float r3 = fmaf(q - al, 549755813888.f, MAGIC);                     // 2^39
        const int G = (__float_as_int(r3) - MAGIC_BITS) - (__float_as_int(r2) - MAGIC_BITS) -
                      ((__float_as_int(r1) - MAGIC_BITS) << 19);
        const uint64_t V = table[k & 127];
        const uint64_t p = V + uint64_t((int64_t(int(V >> 30)) * G) >> 9);        // units of 2^-60
        const int sh = 60 - FRAC + (k >> 7);
        const uint64_t w = (p + (1ull << (sh - 1))) >> (sh & 63);
        return yh < 46.f ? w : 0;                          // below half a unit (l = -inf too)
    }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// x 2^bits, 0 <= x <= 1, rounded down (or up); without fp64, whose unit serves two lanes a cycle.
__device__ __forceinline__ uint64_t fixed(float x, int bits, bool up) {
    const uint32_t b = __float_as_uint(x), e = max(b >> 23, 1u), m = b >> 23 ? (b & 0x7FFFFFu) | 0x800000u : b;
    const int shift = int(e) - 150 + bits;
    if (shift >= 0) return uint64_t(m) << shift;
    if (shift < -24) return up && m ? 1ull : 0ull;
    return (m + (up ? (1u << -shift) - 1u : 0u)) >> -shift;
}
// w / total <= 1 to fp32's rounding: the quotient of both rounded, and what the roundings left.
__device__ __forceinline__ float ratio(uint64_t w, uint64_t total) {
    const float fw = __ull2float_rn(w), ft = __ull2float_rn(total), q = fw / ft;
    const float rw = __ll2float_rn(int64_t(w - __float2ull_rn(fw))), rt = __ll2float_rn(int64_t(total - __float2ull_rn(ft)));
    return q + (fmaf(-q, ft, fw) + fmaf(-q, rt, rw)) / ft;
}

// Bin of y: its sixteenths, rounded down (the addition of 2^23 does that), the last
// bin for all from 1023 / 16 on (and for NaN, an infinite distance at an infinite T).
__device__ __forceinline__ int bin_of(float y) {
    return __float_as_int(__fadd_rd(fminf(y * 16.f, float(NB - 1)), 8388608.f)) - 0x4B000000;
}

template <int T, int C>
__global__ void __launch_bounds__(NT, 2) sample_kernel(const SampleArgs A, const int S) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    float* x = reinterpret_cast<float*>(smem_raw + (sizeof(Shared) + 15) / 16 * 16);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = C > 1 ? int(cl.block_rank()) : 0;
    const int row = int(blockIdx.x) / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s0 = min(rank * S, A.vocab), n = min(S, A.vocab - s0);
    int ex = 0;   // exchange number: its values stay put for three more exchanges
    auto sync = [&]() { if (C > 1) cl.sync(); else __syncthreads(); };

    // ---- read the slice, its maximum
    float mx = -INFINITY;
    {
        const int64_t base = int64_t(row) * A.row_stride + s0;
        constexpr int W = T == 2 ? 4 : 8;          // elements of 16 bytes
        const uint8_t* src = static_cast<const uint8_t*>(A.logits) + base * (16 / W);
        const int nv = (reinterpret_cast<uintptr_t>(src) & 15u) ? 0 : n / W;
        auto put = [&](int i, const uint4& w) {
            float v[W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                v[j] = to_float<T>(&w, j);
                if (v[j] != v[j]) v[j] = -INFINITY;
                mx = fmaxf(mx, v[j]);
            }
#pragma unroll
            for (int j = 0; j < W; j += 4) *reinterpret_cast<float4*>(x + i * W + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        };
        int i = tid;
        for (; i + 3 * NT < nv; i += 4 * NT) {      // four loads in flight
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const uint4*>(src) + i + j * NT);
#pragma unroll
            for (int j = 0; j < 4; ++j) put(i + j * NT, w[j]);
        }
        for (; i < nv; i += NT) put(i, __ldg(reinterpret_cast<const uint4*>(src) + i));
        for (int i = nv * W + tid; i < n; i += NT) {
            float v = to_float<T>(A.logits, base + i);
            if (v != v) v = -INFINITY;
            x[i] = v;
            mx = fmaxf(mx, v);
        }
        if (tid < 128) sh.table[tid] = kPow2.v[tid];
        if (tid == 0) {
            const float t = A.temperature ? A.temperature[row] : 1.f;
            const double c = fmin(1.4426950408889634074 / double(t), 3.0e38);
            sh.chi = float(c);
            sh.clo = float(c - double(float(c)));
        }
    }
    mx = kie::warp_max(mx);
    if (lane == 0) sh.wmax[warp] = __float_as_uint(mx);
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < NWARP; ++w) mx = fmaxf(mx, __uint_as_float(sh.wmax[w]));
        sh.xch[ex][0] = __float_as_uint(mx);
    }
    sync();
    mx = -INFINITY;
#pragma unroll
    for (int r = 0; r < C; ++r) mx = fmaxf(mx, __uint_as_float(uint32_t(cl.map_shared_rank(&sh, r)->xch[ex][0])));
    ex = (ex + 1) & 3;

    const float temp = A.temperature ? A.temperature[row] : 1.f;
    if (mx == -INFINITY) {               // nothing to choose from
        if (rank == 0 && tid == 0) {
            A.tokens[row] = -1;
            if (A.next) A.next[row] = 0;
            if (A.probs) A.probs[row] = 0.f;
        }
        sync();
        return;
    }
    if (!(temp > 0.f)) {                 // greedy: the lowest index of the largest logit
        uint32_t at = 0xFFFFFFFFu;
        for (int i = tid; i < n; i += NT) if (x[i] == mx) { at = uint32_t(s0 + i); break; }
        at = __reduce_min_sync(0xffffffffu, at);
        __syncthreads();
        if (lane == 0) sh.wmin[warp] = at;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < NWARP; ++w) at = min(at, sh.wmin[w]);
            sh.xch[ex][0] = at;
        }
        sync();
        if (rank == 0 && tid == 0) {
            for (int r = 1; r < C; ++r) at = min(at, uint32_t(cl.map_shared_rank(&sh, r)->xch[ex][0]));
            A.tokens[row] = int32_t(at);
            if (A.next) A.next[row] = int32_t(at);
            if (A.probs) A.probs[row] = 1.f;
        }
        sync();
        return;
    }
    if (mx == INFINITY) {                // infinite logits share the mass
        for (int i = tid; i < n; i += NT) x[i] = x[i] == INFINITY ? 0.f : -INFINITY;
        mx = 0.f;
        __syncthreads();
    }
    const Row R{mx, sh.chi, sh.clo, sh.table};

    // Sum over the CTA's threads, for all of them; exclusive prefix and total of it.
    auto block_sum = [&](uint64_t v) {
        v = warp_sum64(v);
        __syncthreads();
        if (lane == 0) sh.wsum[warp] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < NWARP; ++w) v += sh.wsum[w];
        return v;
    };
    auto block_prefix = [&](uint64_t v, uint64_t& total) {
        uint64_t inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        __syncthreads();
        if (lane == 31) sh.wsum[warp] = inc;
        __syncthreads();
        uint64_t before = inc - v;
        total = 0;
#pragma unroll
        for (int w = 0; w < NWARP; ++w) {
            before += w < warp ? sh.wsum[w] : 0ull;
            total += sh.wsum[w];
        }
        return before;
    };

    const int top_k = A.top_k ? A.top_k[row] : 0;
    const float top_p = A.top_p ? A.top_p[row] : 1.f;
    const bool use_k = top_k > 0 && top_k < A.vocab, use_p = top_p < 1.f;

    const float min_p = A.min_p ? A.min_p[row] : 0.f;
    const uint64_t wmin = min_p > 0.f ? fixed(fminf(min_p, 1.f), FRAC, true) : 0ull;
    // warp `warp` holds elements [i0, i1) of the slice where order matters
    const int per = (n + NWARP * 32 - 1) / (NWARP * 32) * 32;
    const int i0 = min(n, warp * per), i1 = min(n, i0 + per);

    constexpr int ABOVE = -2, BELOW = -3;
    // Histogram of the elements for which binf gives a bin (>= 0), summed over the
    // cluster: afterwards each CTA holds its share of the sums in fc/fm[which] and,
    // where `sums` asks for it, the masses of what binf calls ABOVE and BELOW are in
    // above and below.
    // `mine` is then this thread's part, over its warp's range of the slice, of what is
    // above and not cut by min-p.
    uint64_t above = 0, below = 0, mine = 0;
    auto histogram = [&](int which, auto binf, auto sums) {
        for (int i = tid; i < 4 * NB; i += NT) (&sh.h[0][0])[i] = 0u;
        __syncthreads();
        uint64_t sa = 0, sb = 0;
        for (int i = i0 + lane; i < i1; i += 32) {
            const float l = x[i];
            const int b = binf(l);
            if (b >= 0 || (sums.value && b != -1)) {
                const uint64_t w = R.weight(l);
                if (sums.value && b < 0) {
                    sa += b == ABOVE ? w : 0ull;
                    sb += b == ABOVE ? 0ull : w;
                    mine += b == ABOVE && w >= wmin ? w : 0ull;
                } else {
                    atomicAdd(&sh.h[0][b], 1u);
                }
                if (w && b >= 0) {
                    atomicAdd(&sh.h[1][b], uint32_t(w) & 0x7FFFu);
                    atomicAdd(&sh.h[2][b], uint32_t(w >> 15) & 0x7FFFu);
                    atomicAdd(&sh.h[3][b], uint32_t(w >> 30));
                }
            }
        }
        if (sums.value) {
            sa = block_sum(sa);
            sb = block_sum(sb);
            if (tid == 0) { sh.xch[ex][0] = sa; sh.xch[ex][1] = sb; }
        }
        sync();
        if (sums.value) {
            above = below = 0;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                above += cl.map_shared_rank(&sh, r)->xch[ex][0];
                below += cl.map_shared_rank(&sh, r)->xch[ex][1];
            }
            ex = (ex + 1) & 3;
        }
        const int per = NB / C;
        for (int i = tid; i < per; i += NT) {
            const int b = rank * per + i;
            uint32_t cnt = 0;
            uint64_t ms = 0;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const Shared* o = cl.map_shared_rank(&sh, r);
                cnt += o->h[0][b];
                ms += uint64_t(o->h[1][b]) + (uint64_t(o->h[2][b]) << 15) + (uint64_t(o->h[3][b]) << 30);
            }
            sh.fc[which][b] = cnt;
            sh.fm[which][b] = ms;
        }
        sync();
    };
    // The bin of a summed histogram in which the running count (by_mass: mass)
    // reaches `target`; what precedes it and what it holds go to sh.f_*.
    auto find = [&](int which, bool by_mass, uint64_t target, uint32_t cnt0, uint64_t mass0) {
        const Shared* o = cl.map_shared_rank(&sh, (2 * tid) / (NB / C));
        const uint32_t c0 = o->fc[which][2 * tid], c1 = o->fc[which][2 * tid + 1];
        const uint64_t m0 = o->fm[which][2 * tid], m1 = o->fm[which][2 * tid + 1];
        uint32_t ci = c0 + c1;
        uint64_t mi = m0 + m1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t cy = __shfl_up_sync(0xffffffffu, ci, d);
            const uint64_t my = __shfl_up_sync(0xffffffffu, mi, d);
            if (lane >= d) { ci += cy; mi += my; }
        }
        __syncthreads();                 // the last find's results and sums have been read
        if (lane == 31) { sh.wcnt[warp] = ci; sh.wsum[warp] = mi; }
        __syncthreads();
        uint32_t cb = cnt0 + ci - (c0 + c1);
        uint64_t mb = mass0 + mi - (m0 + m1);
        for (int w = 0; w < warp; ++w) { cb += sh.wcnt[w]; mb += sh.wsum[w]; }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t cj = j ? c1 : c0;
            const uint64_t mj = j ? m1 : m0;
            const uint64_t before = by_mass ? mb : cb, with = by_mass ? mb + mj : uint64_t(cb) + cj;
            if (before < target && target <= with) {
                sh.f_bin = 2 * tid + j;
                sh.f_cnt = cb;
                sh.f_mass = mb;
                sh.f_n = cj;
            }
            cb += cj;
            mb += mj;
        }
        __syncthreads();
    };
    // The shortest prefix whose count (mass) reaches target: it ends with the
    // n_eq lowest-indexed of the all_eq tokens of logit of_key(key).
    auto select = [&](bool by_mass, uint64_t target, uint64_t mass0) {   // mass0: before the first histogram
        find(0, by_mass, target, 0u, mass0);
        const int b = sh.f_bin;
        uint32_t cnt = sh.f_cnt;
        uint64_t mass = sh.f_mass;
        // the keys that the bin can hold: its ends in logits, a hundredth of a bin and
        // two neighbours wider than the rounding of y and of the ends can reach
        const float wide = 1.f / (16.f * R.chi);
        uint32_t hi = key_of<T>(R.m - (float(b) - 0.01f) * wide), lo = b == NB - 1 ? 0u : key_of<T>(R.m - (float(b) + 1.01f) * wide);
        hi = min(hi, key_of<T>(R.m) - 2u) + 2u;
        lo = max(lo, 2u) - 2u;
        for (int level = 0; level < 4; ++level) {    // 2^32 -> 2^22 -> 2^12 -> 2^2 -> 1 keys
            int shift = 0;
            while (shift < 22 && ((hi - lo) >> shift) >= NB) ++shift;
            auto here = [&](float l) {
                const uint32_t k = key_of<T>(l);
                if (bin_of(R.y(l)) != b || (level > 0 && (k < lo || k > hi))) return -1;   // the keys reach over the bin's ends
                return int(min((hi - min(k, hi)) >> shift, uint32_t(NB - 1)));
            };
            histogram(1, here, std::false_type());
            find(1, by_mass, target, cnt, mass);
            const int s = sh.f_bin;
            const uint32_t nc = sh.f_n;
            cnt = sh.f_cnt;
            mass = sh.f_mass;
            if (shift == 0) {
                if (tid == 0) {
                    hi -= uint32_t(s);
                    const uint64_t w = R.weight(of_key<T>(hi));
                    const uint64_t need = by_mass ? (w ? (target - mass + w - 1) / w : nc) : target - cnt;
                    sh.key = hi;
                    sh.all_eq = nc;
                    sh.n_eq = uint32_t(need < nc ? need : nc);
                    sh.mass = mass + sh.n_eq * w;
                }
                __syncthreads();
                return;
            }
            if (nc > LIST) {           // many near-equal logits: into the bucket's keys
                hi -= uint32_t(s) << shift;
                lo = max(lo, hi - ((1u << shift) - 1u));
                continue;
            }
            if (tid == 0) sh.list_n = 0;
            __syncthreads();
            for (int i = tid; i < n; i += NT)
                if (here(x[i]) == s) {
                    const uint32_t at = atomicAdd(&sh.list_n, 1u);
                    sh.list_key[at] = key_of<T>(x[i]);
                    sh.list_idx[at] = s0 + i;
                    sh.list_w[at] = R.weight(x[i]);
                }
            sync();
            if (warp == 0) {
                uint32_t key = 0u;
                int32_t idx = 0x7FFFFFFF;
                uint64_t w = 0;
                int k = lane;
#pragma unroll
                for (int r = 0; r < C; ++r) {
                    const Shared* o = cl.map_shared_rank(&sh, r);
                    const int m = int(o->list_n);
                    if (k >= 0 && k < m) { key = o->list_key[k]; idx = o->list_idx[k]; w = o->list_w[k]; k = -1; }
                    else if (k >= 0) k -= m;
                }
                const bool have = idx != 0x7FFFFFFF;
                uint32_t before = 0, eq = 0, eq_all = 0;
                uint64_t mb = 0;
                for (int j = 0; j < 32; ++j) {
                    const uint32_t kj = __shfl_sync(0xffffffffu, key, j);
                    const int32_t ij = __shfl_sync(0xffffffffu, idx, j);
                    const uint64_t wj = __shfl_sync(0xffffffffu, w, j);
                    if (ij == 0x7FFFFFFF) continue;
                    if (kj > key || (kj == key && ij < idx)) { ++before; mb += wj; }
                    if (kj == key) { ++eq_all; if (ij <= idx) ++eq; }
                }
                const uint64_t with = by_mass ? mass + mb + w : uint64_t(cnt) + before + 1;
                const uint64_t without = by_mass ? mass + mb : uint64_t(cnt) + before;
                // equal masses before and after (w = 0) cannot both straddle the target
                if (have && without < target && target <= with) {
                    sh.key = key;
                    sh.n_eq = eq;
                    sh.all_eq = eq_all;
                    sh.mass = mass + mb + w;
                }
            }
            sync();                      // the lists may be written again
            return;
        }
    };

    const float uf = A.u[row];
    const uint64_t U = uf >= 1.f ? ~0ull : uf > 0.f ? fixed(uf, 64, false) : 0ull;
    // the least mass that is at least p of `mass`, and at least one token's
    auto p_target = [&](uint64_t mass) {
        const uint64_t P = top_p > 0.f ? fixed(top_p, 64, false) : 0ull;
        const uint64_t t = __umul64hi(mass, P) + (mass * P != 0ull ? 1ull : 0ull);
        return t ? t : 1ull;
    };
    auto choose = [&](int token, uint64_t w, uint64_t total) {
        A.tokens[row] = token;
        if (A.next) A.next[row] = token;
        if (A.probs) A.probs[row] = ratio(w, total);
    };
    // Where the running sum of val(bin, words summed over the cluster) over the bins of the
    // single-word histogram `hist` reaches the targets aim(sum of all): the bins go to f_bin
    // and f_n, the running sum with the first of them to f_mass.  Each CTA sums its share of
    // the bins (every CTA reading all of 4,096 bins of 8 CTAs took 7 us).  The bin beyond the
    // last stands for a target that is not reached.
    auto crossing = [&](const uint32_t* hist, auto bins, auto val, auto aim) {
        constexpr int N = decltype(bins)::value, PER = N / C, PT = PER > NT ? PER / NT : 1;
        const int at = tid * PT, bin = rank * PER + at;
        if (tid == 0) { sh.f_bin = N; sh.f_n = N; sh.f_mass = ~0ull; }
        sync();
        uint64_t q[PT], qs = 0, all;
#pragma unroll
        for (int j = 0; j < PT; ++j) q[j] = 0;
        if (at < PER) {
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const uint32_t* o = cl.map_shared_rank(const_cast<uint32_t*>(hist), r) + bin;
#pragma unroll
                for (int j = 0; j < PT; ++j) q[j] += o[j];
            }
#pragma unroll
            for (int j = 0; j < PT; ++j) {
                q[j] = val(bin + j, q[j]);
                qs += q[j];
            }
        }
        uint64_t before = block_prefix(qs, all);
        if (tid == 0) sh.xch[ex][0] = all;
        sync();
        all = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const uint64_t v = cl.map_shared_rank(&sh, r)->xch[ex][0];
            before += r < rank ? v : 0ull;
            all += v;
        }
        ex = (ex + 1) & 3;
        const ulonglong2 t = aim(all);
        if (at < PER) {
#pragma unroll
            for (int j = 0; j < PT; ++j) {
                const uint64_t with = before + q[j];
                if (before < t.x && t.x <= with)
                    for (int r = 0; r < C; ++r) { Shared* o = cl.map_shared_rank(&sh, r); o->f_bin = bin + j; o->f_mass = with; }
                if (before < t.y && t.y <= with)
                    for (int r = 0; r < C; ++r) cl.map_shared_rank(&sh, r)->f_n = uint32_t(bin + j);
                before = with;
            }
        }
        sync();
    };
    // Bitonic sort of fm[1][0 .. np) (np a power of two from 64 to CAP), ascending.
    auto sort = [&](int np) {
        for (int k = 2; k <= np; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                if (tid < np / 2) {
                    const int i = ((tid & ~(j - 1)) << 1) | (tid & (j - 1));
                    const uint64_t lo = sh.fm[1][i], hi = sh.fm[1][i | j];
                    if ((lo > hi) == ((i & k) == 0)) { sh.fm[1][i] = hi; sh.fm[1][i | j] = lo; }
                }
                // a warp's 32 pairs of a step j <= 32 are its own 64 elements; the next step's too
                // unless it is a longer one
                if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
                else __syncwarp();
            }
        __syncthreads();
    };

    uint64_t* list = reinterpret_cast<uint64_t*>(sh.h[2]);   // CAP candidates, once the histogram has been summed
    if (use_k && top_k <= KLIM) {
        // ---- sorted path: the bins that hold the first top_k tokens go to CTA 0
        uint32_t* hist = sh.h[0];
        for (int i = tid; i < NB; i += NT) hist[i] = 0u;
        __syncthreads();
        for (int i = tid; i < n; i += NT) atomicAdd(&hist[bin_of(R.y(x[i]))], 1u);
        crossing(hist, std::integral_constant<int, NB>(), [](int, uint64_t v) { return v; },
                 [&](uint64_t) { return ulonglong2{uint64_t(top_k), uint64_t(top_k)}; });
        const int b = sh.f_bin, nc = sh.f_mass <= CAP ? int(sh.f_mass) : CAP + 1;
        if (nc <= CAP) {
            // this CTA's candidates in index order; bin <= b: 16 y below b + 1
            const float yend = b < NB - 1 ? float(b + 1) : INFINITY;
            auto in_bins = [&](float l) { return R.y(l) * 16.f < yend || b == NB - 1; };
            uint32_t cw = 0, base = 0, own = 0;
            for (int i = i0 + lane; i < i1; i += 32) cw += in_bins(x[i]);
            cw = __reduce_add_sync(0xffffffffu, cw);
            if (lane == 0) sh.wcnt[warp] = cw;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < NWARP; ++w) {
                base += w < warp ? sh.wcnt[w] : 0u;
                own += sh.wcnt[w];
            }
            for (int i = i0; cw && i < i1; i += 32) {
                const float l = i + lane < i1 ? x[i + lane] : 0.f;
                const bool in = i + lane < i1 && in_bins(l);
                const uint32_t hit = __ballot_sync(0xffffffffu, in);
                if (in) list[base + __popc(hit & ((1u << lane) - 1u))] = uint64_t(key_of<T>(l)) << 32 | uint32_t(s0 + i + lane);
                base += __popc(hit);
            }
            if (tid == 0) sh.xch[ex][0] = own;
            sync();
            if (rank != 0) {
                cl.barrier_arrive();
                cl.barrier_wait();       // CTA 0 has read the list
                return;
            }
            int cnt[C];
#pragma unroll
            for (int r = 0; r < C; ++r) cnt[r] = int(cl.map_shared_rank(&sh, r)->xch[ex][0]);
            int np = 64;
            while (np < nc) np *= 2;
            for (int i = tid; i < np; i += NT) {
                uint64_t v = 0;
                int at = i;
#pragma unroll
                for (int r = 0; r < C; ++r) {
                    if (at >= 0 && at < cnt[r]) v = cl.map_shared_rank(list, r)[at];
                    at = at < cnt[r] ? -1 : at - cnt[r];
                }
                if (i < nc) {
                    const uint32_t k = uint32_t(v >> 32);
                    sh.fc[1][i] = uint32_t(v);
                    sh.fm[0][i] = R.weight(of_key<T>(k));
                    sh.fm[1][i] = uint64_t(~k) << 32 | uint32_t(i);
                } else sh.fm[1][i] = ~0ull;
            }
            if (C > 1) cl.barrier_arrive();
            __syncthreads();
            sort(np);
            int pos[2];
            uint64_t w[2], total;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = 2 * tid + j;
                pos[j] = i < nc ? int(uint32_t(sh.fm[1][i])) : -1;
                w[j] = i < nc && i < top_k ? sh.fm[0][pos[j]] : 0ull;   // the first top_k
            }
            uint64_t mb = block_prefix(w[0] + w[1], total);
            const uint64_t target = use_p ? p_target(total) : ~0ull;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool keep = mb < target && w[j] >= wmin;
                mb += w[j];
                if (pos[j] >= 0) sh.fm[0][pos[j]] = keep ? w[j] : 0ull;
            }
            __syncthreads();
            // the draw, in index order
#pragma unroll
            for (int j = 0; j < 2; ++j) w[j] = 2 * tid + j < nc ? sh.fm[0][2 * tid + j] : 0ull;
            mb = block_prefix(w[0] + w[1], total);
            const uint64_t draw = __umul64hi(total, U);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (mb <= draw && draw < mb + w[j]) choose(int(sh.fc[1][2 * tid + j]), w[j], total);
                mb += w[j];
            }
            if (C > 1) cl.barrier_wait();
            return;
        }
    }

    // ---- the kept prefix: every logit above `key`, and of those equal to it the n_eq lowest-
    // indexed, or all up to index `last`
    uint32_t key = 0u, n_eq = 0xFFFFFFFFu, all_eq = 0u, last = 0xFFFFFFFFu;
    float counted = -1.f;                // logits of a smaller 16 y are in `mine` already
    bool summed = false;                 // or all are
    if (use_k) {
        histogram(0, [&](float l) { return bin_of(R.y(l)); }, std::false_type());
        select(false, uint64_t(top_k), 0ull);
        __syncthreads();
        const uint64_t mass = sh.mass;
        key = sh.key; n_eq = sh.n_eq; all_eq = sh.all_eq;
        if (use_p) {
            select(true, p_target(mass), 0ull);
            __syncthreads();
            key = sh.key; n_eq = sh.n_eq; all_eq = sh.all_eq;
        }
    } else if (use_p) {
        // masses of the fine bins to 2^-14: 2^(f / 64) in units of 2^-14, f the distance to the bin's end
        uint32_t* hist = &sh.h[0][0];
        for (int i = tid; i < NF; i += NT) hist[i] = 0u;
        if (tid == 0) sh.list_n = 0u;
        __syncthreads();
        for (int i = tid; i < n; i += NT) {
            const float y = R.y(x[i]) * 64.f;
            if (y < 46.f * 64.f) {
                const float down = __fadd_rd(y, 8388608.f);
                float v;                   // in [1, 2^(1/64)]: rounded to 14 fraction bits
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(fmaf(down - 8388608.f - y, 1.f / 64.f, 1.f / 64.f)));
                atomicAdd(&hist[__float_as_int(down) - 0x4B000000], (__float_as_uint(v) - 0x3F000000u + 256u) >> 9);
            }
        }
        // The prefix ends where the mass passes p of the total, both sums of words good to 2^-15 and
        // to y's rounding, 2^-18 of a weight, in units of 2^-40 (2^18 tokens at most): within a
        // 2^-13th of the target.
        crossing(hist, std::integral_constant<int, NF>(),
                 [](int bin, uint64_t v) { return uint64_t(float(v) * exp2f(26.f - float(bin + 1) / 64.f)); },
                 [&](uint64_t total) {
                     const float want = fmaxf(top_p, 0.f) * float(total);
                     return ulonglong2{uint64_t(fmaxf(want * (1.f - 1.f / 8192.f), 1.f)), uint64_t(fmaxf(want * (1.f + 1.f / 8192.f), 1.f))};
                 });
        const int b1 = min(sh.f_bin, NF - 1), b2 = min(int(sh.f_n), NF - 1);
        const float y1 = float(b1), y2 = b2 < NF - 1 ? float(b2 + 1) : INFINITY;    // the bins [b1, b2]: 64 y in [y1, y2)
        // the one exact pass: sums before and after those bins, their tokens to a list
        uint64_t sa = 0, sb = 0;
        for (int i = i0 + lane; i < i1; i += 32) {
            const float l = x[i], y = R.y(l) * 64.f;
            if (y >= y1 && y < y2) {
                const uint32_t at = atomicAdd(&sh.list_n, 1u);
                if (at < CAP) list[at] = uint64_t(~key_of<T>(l)) << 32 | uint32_t(s0 + i);
            } else {
                const uint64_t w = R.weight(l);
                sa += y < y1 ? w : 0ull;
                sb += y < y1 ? 0ull : w;
                mine += y < y1 && w >= wmin ? w : 0ull;
            }
        }
        sa = block_sum(sa);
        sb = block_sum(sb);
        if (tid == 0) { sh.xch[ex][0] = sa; sh.xch[ex][1] = sb; sh.xch[ex][2] = sh.list_n; }
        sync();
        uint64_t head = 0, tail = 0;
        int cnt[C], nc = 0, cnt_own = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const uint64_t* v = cl.map_shared_rank(&sh, r)->xch[ex];
            head += v[0];
            tail += v[1];
            cnt[r] = int(v[2]);
            nc += cnt[r];
            cnt_own = r == rank ? cnt[r] : cnt_own;
        }
        ex = (ex + 1) & 3;
        if (nc <= CAP) {
            if (rank == 0) {
                int np = 64;
                while (np < nc) np *= 2;
                for (int i = tid; i < np; i += NT) {
                    uint64_t v = ~0ull;
                    int at = i;
#pragma unroll
                    for (int r = 0; r < C; ++r) {
                        if (at >= 0 && at < cnt[r]) v = cl.map_shared_rank(list, r)[at];
                        at = at < cnt[r] ? -1 : at - cnt[r];
                    }
                    sh.fm[1][i] = v;
                }
                __syncthreads();
                sort(np);              // logit descending, index ascending
                uint64_t w[2], inside;
                uint32_t k2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = 2 * tid + j;
                    k2[j] = i < nc ? ~uint32_t(sh.fm[1][i] >> 32) : 0u;
                    w[j] = i < nc ? R.weight(of_key<T>(k2[j])) : 0ull;
                }
                uint64_t mb = head + block_prefix(w[0] + w[1], inside);
                const uint64_t target = p_target(head + inside + tail);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (mb < target && target <= mb + w[j]) { sh.key = k2[j]; sh.last = uint32_t(sh.fm[1][2 * tid + j]); }
                    mb += w[j];
                }
            }
            sync();
            const Shared* o = cl.map_shared_rank(&sh, 0);
            key = o->key;
            last = o->last;
            // the kept tokens of this CTA's list, to the sums of their warps' ranges
            if (tid < NWARP) sh.wsum[tid] = 0;
            __syncthreads();
            for (int i = tid; i < cnt_own; i += NT) {
                const uint64_t v = list[i];
                if (v <= (uint64_t(~key) << 32 | last)) {
                    const uint64_t w = R.weight(of_key<T>(~uint32_t(v >> 32)));
                    if (w >= wmin) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.wsum[(int(uint32_t(v)) - s0) / per]), w);
                }
            }
            __syncthreads();
            mine += lane == 0 ? sh.wsum[warp] : 0ull;
            summed = true;
        } else {
            // a crowd: histograms of exact masses
            mine = 0;
            const int c1 = b1 / 4, c2 = b2 / 4;
            counted = float(c1);
            histogram(0, [&](float l) { const int b = bin_of(R.y(l)); return b < c1 ? ABOVE : b > c2 ? BELOW : b; }, std::true_type());
            const uint64_t first = above;
            const Shared* o = cl.map_shared_rank(&sh, (2 * tid) / (NB / C));
            const uint64_t inside = block_sum(o->fm[0][2 * tid] + o->fm[0][2 * tid + 1]);
            select(true, p_target(first + inside + below), first);
            __syncthreads();
            key = sh.key; n_eq = sh.n_eq; all_eq = sh.all_eq;
        }
    }

    // ---- masses in index order
    uint32_t eq0 = 0;                    // equal tokens before this warp's
    const bool ties = n_eq < all_eq;
    if (ties) {
        uint32_t c = 0;
        for (int i = i0 + lane; i < i1; i += 32) c += key_of<T>(x[i]) == key;
        c = __reduce_add_sync(0xffffffffu, c);
        __syncthreads();
        if (lane == 0) sh.wcnt[warp] = c;
        __syncthreads();
        if (tid == 0) {
            uint64_t a = 0;
            for (int w = 0; w < NWARP; ++w) a += sh.wcnt[w];
            sh.xch[ex][1] = a;
        }
        sync();
        for (int r = 0; r < rank; ++r) eq0 += uint32_t(cl.map_shared_rank(&sh, r)->xch[ex][1]);
        for (int w = 0; w < warp; ++w) eq0 += sh.wcnt[w];
        ex = (ex + 1) & 3;
    }
    // past this y a weight is below min_p (half a percent more, for the rounding of both)
    const float ymax = min_p > 0.f ? -log2f(fminf(min_p, 1.f)) * 1.005f + 0.005f : INFINITY;
    // kept mass of element i < end (lanes in index order); eq: equal tokens before this group of 32
    auto kept = [&](int i, int end, uint32_t& eq, float from) -> uint64_t {
        const float l = i < end ? x[i] : -INFINITY;
        const float y = R.y(l);
        const uint32_t k = key_of<T>(l);
        bool keep = i < end && (k > key || (k == key && uint32_t(s0 + i) <= last)) && y < ymax && y * 16.f >= from;
        if (ties) {
            const uint32_t same = __ballot_sync(0xffffffffu, i < end && k == key);
            if (k == key) keep = keep && eq + __popc(same & ((1u << lane) - 1u)) < n_eq;
            eq += __popc(same);
        }
        if (!__any_sync(0xffffffffu, keep)) return 0;
        const uint64_t w = keep ? R.weight(l) : 0;
        return w >= wmin ? w : 0;
    };
    uint64_t sum = mine;
    if (!use_k && !use_p && min_p <= 0.f) {
        for (int i = i0 + lane; i < i1; i += 32) sum += R.weight(x[i]);
    } else if (!summed) {
        uint32_t eq = eq0;
        for (int i = i0; i < i1; i += 32) sum += kept(i + lane, i1, eq, counted);
    }
    sum = warp_sum64(sum);
    __syncthreads();
    if (lane == 0) sh.wsum[warp] = sum;
    if (ties && lane == 0) sh.wmin[warp] = eq0;
    __syncthreads();
    uint64_t cta = 0;
#pragma unroll
    for (int w = 0; w < NWARP; ++w) cta += sh.wsum[w];
    if (tid == 0) sh.xch[ex][2] = cta;
    sync();
    uint64_t total = 0, start = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        const uint64_t v = cl.map_shared_rank(&sh, r)->xch[ex][2];
        if (r < rank) start += v;
        total += v;
    }
    // no CTA leaves while another may read its shared memory: all of that is done here
    if (C > 1) cl.barrier_arrive();
    const uint64_t target = __umul64hi(total, U);
    if (start <= target && target < start + cta) {       // this CTA holds the crossing: all its warps look
        int cw = 0;
        while (start + sh.wsum[cw] <= target) start += sh.wsum[cw++];
        const int c0 = min(n, cw * per), c1 = min(n, c0 + per);          // the crossing warp's range, cut into NWARP
        const int part = (c1 - c0 + NWARP * 32 - 1) / (NWARP * 32) * 32, b0 = min(c1, c0 + warp * part), b1 = min(c1, b0 + part);
        uint32_t eq = ties ? sh.wmin[cw] : 0u;
        if (ties) {                                       // equal tokens before this warp's part
            uint32_t e = 0;
            for (int i = c0 + lane; i < b0; i += 32) e += key_of<T>(x[i]) == key;
            eq += __reduce_add_sync(0xffffffffu, e);
        }
        uint64_t own = 0;
        {
            uint32_t e = eq;
            for (int i = b0; i < b1; i += 32) own += kept(i + lane, b1, e, -1.f);
        }
        own = warp_sum64(own);
        __syncthreads();                                  // the warps' sums have been read
        if (lane == 0) sh.wsum[warp] = own;
        __syncthreads();
        for (int w = 0; w < warp; ++w) start += sh.wsum[w];
        if (start <= target && target < start + own) {
            for (int i = b0; i < b1; i += 32) {
                const uint64_t w = kept(i + lane, b1, eq, -1.f);
                uint64_t inc = w;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint64_t v = __shfl_up_sync(0xffffffffu, inc, d);
                    if (lane >= d) inc += v;
                }
                const uint32_t hit = __ballot_sync(0xffffffffu, start + inc > target);
                if (hit) {
                    if (lane == __ffs(hit) - 1) choose(s0 + i + lane, w, total);
                    break;
                }
                start += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
    }
    if (C > 1) cl.barrier_wait();
}

template <int T, int C>
cudaError_t launch(const SampleArgs& a, int S, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const int smem = int((sizeof(Shared) + 15) / 16 * 16) + S * 4;
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(done.load(std::memory_order_acquire) & bit)) {
        r = cudaFuncSetAttribute(sample_kernel<T, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (r != cudaSuccess) return r;
        if (dev < 64) done.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows) * C);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T, C>, a, S);
}

template <int T>
cudaError_t launch_t(const SampleArgs& a, int C, int S, cudaStream_t st) {
    if (C == 1) return launch<T, 1>(a, S, st);
    if (C == 2) return launch<T, 2>(a, S, st);
    if (C == 4) return launch<T, 4>(a, S, st);
    return launch<T, 8>(a, S, st);
}

}  // namespace

extern "C" cudaError_t kie_launch_sample(const SampleArgs* a, int sms, cudaStream_t st) {
    // CTAs per row: while one per SM is left over and a slice is above 4,096, and at least
    // so many that a slice fits shared memory.  Top-p 0.9 with 1, 2, 4, 8 CTAs a row, us:
    // 1 x 4,000 15.1, 16.2, 15.6, 16.9; 1 x 32,000 35, 27, 21, 20; 32 x 32,000 37, 28, 22,
    // 27; 64 x 32,000 37, 29, 28, 50; 256 x 32,000 72, 74, 93, 179.
    int C = 1;
    while (C < MAXC && ((int64_t(a->rows) * 2 * C <= sms && a->vocab > C * 4096) || int64_t(a->vocab) > int64_t(C) * 32768)) C *= 2;
    const int S = ((a->vocab + C - 1) / C + 7) / 8 * 8;
    if (a->type == 0) return launch_t<0>(*a, C, S, st);
    if (a->type == 1) return launch_t<1>(*a, C, S, st);
    return launch_t<2>(*a, C, S, st);
}
