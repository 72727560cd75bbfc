// extend_tc.cuh -- attention of several new tokens per sequence on the tensor
// cores (16-bit pools).
//
// Mathematics as in extend_fma_f32.cu: one pass over the keys that a tile of 128
// query rows sees, with a running reference m and sum l per row,
//   S = Q K^T,  P = 2^(f(S) - m),  O += P V,  l += sum P,  out = O / l.
// S and O live in TMEM.  The softmax reads a row of S, writes P over it in the
// pool's type, and P is the A operand of P V straight from TMEM.  m is set by the
// row's first scores and moves only when a later one passes it by 2^8, so O is
// rarely rescaled.
//
// Roles in a CTA: one warp stages K and V (TMA, 16-row runs of the pages, a
// ring of tiles), one thread per row tile issues the products, four warps per
// row tile do the softmax, a row to a thread.  They meet at mbarriers; every
// wait is bounded.
//
// What bounds it, as measured:
//   - few rows, long ranges (single tokens, trees): HBM.  64 single tokens over
//     512-8192 with 256-wide heads and capped scores 328 us, 6.9 TB/s; 32 trees
//     of up to 32 nodes over 512-8192 108 us, 5.4 TB/s (6.1 in the kernel; the
//     rest is the joining pass and the CTAs' ends).
//   - many rows: softmax and products of a row tile follow each other, and two
//     row tiles share an SM.  Three prompts of 2048-6144 tokens, 32 heads of
//     128: 381 us, 1.26 PFLOP/s, tensor pipe 57 % busy.  Per 128 keys and row
//     tile the softmax takes 1700 cycles (two readings of the scores 600, the
//     exponentials 1000) and the products 1300 at the rate that a large GEMM
//     reaches; the first half of P V runs beside the softmax.
//   - capped or biased scores: the softmax's arithmetic (FMA pipe 32 % busy,
//     issue slots 45 %, two softmax warps per scheduler): 64 keys take 2000
//     cycles a warp, 1000-1200 of them in capping and masking.  24 sequences
//     with capped scores in a window of 1024 180 us, tensor pipe 33 %.
//   - small calls: a CTA's start (2000-3500 cycles to its item, 4000 more to its
//     first scores) and its end (2500).
#pragma once

#include "extend_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

constexpr float kTcLog2e = 1.4426950408889634f;
// A row's reference is its first maximum, so that a row that sees one key has
// the weight 1 and gets that value bit by bit; it moves once a score passes it by
// 2^8.  In fp16, whose small weights have fewer bits, it lies 2^7 lower, which is
// exact as well: largest weights are 2^7 to 2^15, and bits go from 2^-21 of the
// largest on, not from 2^-14.
template <bool BF16>
struct TcRef {
    static constexpr float kBelow = BF16 ? 0.f : 7.f;
    static constexpr float kLag = BF16 ? 8.f : 15.f;
};

// NQ tiles of 128 rows share each staged tile of K and V.  One: two CTAs per
// SM, whose loads, products and softmax overlap each other (D = 256 has room
// for one).  Two, at D = 128: one CTA per SM, its two row tiles in turn on the
// tensor cores and in softmax, for half the L2 reads per row and a deeper ring.
template <int D, int NQ>
struct TcShape {
    static constexpr int KT = NQ == 1 ? 64 : 128;       // keys of a staged tile
    static constexpr int NS = NQ == 1 ? 2 : 1;          // score tiles of a row tile in TMEM
    // rings of K and of V tiles, as many as fit beside the queries
    static constexpr int NK = D == 64 ? 4 : D == 128 && NQ == 1 ? 2 : 3;
    static constexpr int NV = D == 64 ? 4 : D == 128 && NQ == 1 ? 3 : 2;
    static constexpr int kCtas = D == 256 || NQ == 2 ? 1 : 2;  // per SM
    static constexpr int kRows = NQ * 128;
    static constexpr int kSlabs = D / 64;               // 128-byte slabs of a row
    static constexpr int kTileBytes = KT * D * 2;
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kOCol = NQ * NS * KT;          // TMEM columns: scores, then outputs
    static constexpr int kCols = kOCol + NQ * D <= 256 ? 256 : 512;
    static constexpr int kThreads = kRows + 32 + NQ * 32;
    static constexpr int kTiles = NQ * kQBytes + (NK + NV) * kTileBytes;  // then TcControl
    static_assert(kOCol + NQ * D <= 512, "TMEM columns");
    // the product warps' order: score tiles ahead of one row tile's outputs, or two row
    // tiles in turn with one score tile each
    static_assert((NQ == 1 && NS == 2) || (NQ == 2 && NS == 1), "score tiles");
};

struct TcControl {
    uint64_t full[8], empty[8],  // the rings': K tiles, then V tiles
        q_full, s_full[2], p_half[2], p_ready[2], o_full[2], o_last[2], turn[2];
    uint32_t tmem;
    volatile int stop;  // a wait ran past its bound
    uint32_t bad[8];    // runs of recent tiles that no row sees (one bit each)
    ExtTile tile;       // the CTA's item
    int part;
    // What the tile's edges are told by; kept here, not in registers, between them.
    int base;               // position of the sequence's first new token
    int ntok, q0, prefix;
    int k0, k1, kmin;       // the part's keys; first key that some row sees
    int same_lo, same_hi;   // keys that every row sees
    int inner_lo, inner_hi; // ... of those in the part
};

// Bounded wait: false once it, or any other wait of the CTA, has given up.
// The timer is slow to read (hundreds of cycles, in which a barrier that has
// completed goes unseen), so it is first looked at after many tries.
__device__ __forceinline__ bool tc_wait(TcControl &c, uint64_t *bar, unsigned parity,
                                        int32_t *dev_error) {
    unsigned long long t0 = 0;
    for (unsigned it = 0; !mbar_try_wait(bar, parity); ++it) {
        if ((it & 255u) != 255u) continue;
        if (c.stop) return false;
        const unsigned long long now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            c.stop = 1;
            raise_fault(dev_error, PKV_FAULT_TIMEOUT);
            return false;
        }
    }
    return true;
}

// Bits [lo, hi) of a 32-bit word, the bounds taken within it.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
    lo = max(lo, 0), hi = min(hi, 32);
    if (hi <= lo) return 0;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Which of the 32 keys from k + 32 * word on a row sees: those in [lo, hi), and
// in a tree those nodes in its mask `words`.  `bad` are the tile's runs that no
// row sees.
__device__ __forceinline__ uint32_t tc_seen(const ExtArgs &a, const TcControl &c, int lo, int hi,
                                            const uint32_t *words, int k, int word, uint32_t bad) {
    const int b = k + word * 32;
    uint32_t see = bit_range(lo - b, hi - b);
    if (words) {
        const int n0 = b - c.base, w0 = n0 >> 5, sh = n0 & 31;
        if (n0 + 31 >= 0 && n0 < c.ntok) {
            uint32_t x = 0;
            if (w0 >= 0) x = __ldg(words + w0) >> sh;
            if (sh && w0 + 1 < a.mask_words) x |= __ldg(words + w0 + 1) << (32 - sh);
            see |= x & bit_range(-n0, c.ntok - n0);
        }
    }
    if ((bad >> (2 * word)) & 1u) see &= 0xffff0000u;
    if ((bad >> (2 * word + 1)) & 1u) see &= 0x0000ffffu;
    return see;
}

// Rows of a tile of V that no row of the CTA sees count with weight zero, and
// what lies there may not be finite: they are cleared.  Thread i of n.
template <int D, int KT>
__device__ __forceinline__ void tc_clear_values(unsigned char *tile, int lo, int hi, uint32_t bad, int i, int n) {
    constexpr int C = D / 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto at = [&](int x) { return reinterpret_cast<uint4 *>(tile + swz_offset<KT>(x / C, x % C)); };
    for (int x = i; x < lo * C; x += n) *at(x) = zero;
    for (int x = hi * C + i; x < KT * C; x += n) *at(x) = zero;
    for (; bad; bad &= bad - 1) {
        const int r = __ffs(bad) - 1;  // a run
        for (int x = r * kExtRun * C + i; x < (r + 1) * kExtRun * C; x += n) *at(x) = zero;
    }
    fence_proxy_async_smem();
}

// Results that are not finite.  The product gives a value at a key that a row does
// not see, and others of its tile do, the weight zero, and 0 * inf is NaN: a row's
// NaN may not be its own.  It is where the sum l is NaN (a score that the row sees
// was).  Where l is a number and a result is not finite, the part's values are looked
// at, and rows whose result may not be their own are computed again.

// Of one run of keys (16 rows of D values), those with a value that is not finite,
// and 16 bits further up those with an infinite one.  By a whole warp.
template <typename T, int D>
__device__ __forceinline__ uint32_t tc_odd_keys(const T *run) {
    constexpr uint32_t kInf = __is_same(T, __nv_bfloat16) ? 0x7f80u : 0x7c00u;
    const int lane = threadIdx.x & 31;
    uint4 v[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(run) + i * 32 + lane);
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        bool any = false, inf = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
            any |= lo >= kInf || hi >= kInf;
            inf |= lo == kInf || hi == kInf;
        }
        odd |= ((any ? 1u : 0u) | (inf ? 0x10000u : 0u)) << ((i * 32 + lane) / (D / 8));
    }
    return __reduce_or_sync(0xffffffffu, odd);
}

// Whether the lane's row has to be computed again (1; 2: with small weights); `nan`: it has a NaN, `inf`: it has
// an infinity (or nearly) and no NaN.  lo, hi and words: what it sees, as in tc_seen.
//   - A NaN is the row's own if it sees a NaN, and no value that is not finite lies at
//     a key that it does not see, nor an infinite one at a key that it does (a weight
//     that rounds to zero, or has no remainder, makes NaN of it).
//   - An infinity is its own if it sees one: from another key it would be a NaN.
//   - Either may come from finite values whose sum passes fp32's range, since the
//     weights' sum is above 1.  Smaller weights, whose sum is not, keep it within.
template <typename T, int D>
__device__ __noinline__ int tc_not_its_own(const ExtArgs &a, const TcControl &c, int seq, int kvh, bool nan,
                                            bool inf, int lo, int hi, const uint32_t *words) {
    const int32_t *tbl = a.block_tables + (size_t)seq * a.max_blocks_per_seq;
    const int first = max(c.k0, c.kmin);  // what lies before was cleared
    bool sees_nan = false, sees_inf = false, other = false;
    for (int k = first & ~(kExtRun - 1); k < c.k1; k += kExtRun) {
        const int run = k / kExtRun, blk = __ldg(tbl + (run >> a.run_shift));
        if (blk < 0 || blk >= a.num_blocks) continue;
        const size_t row = ((((size_t)blk * a.num_kv_heads + kvh) << a.run_shift) + (run & ((1 << a.run_shift) - 1))) * kExtRun;
        const uint32_t odd = tc_odd_keys<T, D>(static_cast<const T *>(a.v_pool) + row * D);
        if (odd == 0) continue;
        const uint32_t part = bit_range(first - k, c.k1 - k), see = tc_seen(a, c, lo, hi, words, k, 0, 0);
        sees_nan |= (odd & part & see & 0xffffu) != 0;
        sees_inf |= ((odd >> 16) & part & see) != 0;
        other |= (odd & part & ~see & 0xffffu) != 0;
        // all is known
        if (__all_sync(0xffffffffu, nan ? other || sees_inf : !inf || sees_inf)) break;
    }
    if (nan ? sees_nan && !sees_inf && !other : !inf || sees_inf) return 0;
    return sees_nan || sees_inf || other ? 1 : 2;
}

// Rows first + i of a tile, for the bits i of `rows`, again, one at a time on the
// CUDA cores, straight from the pool, by the warp that has written them: a key to a
// lane for the scores, then the columns to the lanes for the values.  Those of
// `small` with weights 2^-24 times as large.
template <typename T, int D>
__device__ __noinline__ void tc_redo_rows(const ExtArgs &a, ExtTile t, int kvh, int k0, int k1,
                                          int part, int first, uint32_t rows, uint32_t small) {
    constexpr int PER = D / 32, kVec = 8;
    const int lane = threadIdx.x & 31, G = a.group;
    for (; rows; rows &= rows - 1) {
        const int row = t.row0 + first + __ffs(rows) - 1, tok = row / G, h = kvh * G + row - tok * G;
        const size_t oh = (size_t)(t.q0 + tok) * a.num_heads + h;
        const int pos = t.ctx - t.ntok + tok, base = t.ctx - t.ntok;
        int lo = 0, hi = base;
        if (!a.tree_mask) ext_row_range(a, t.prefix, pos, lo, hi);
        const float slope = a.slopes ? __ldg(a.slopes + h) * kTcLog2e : 0.f;
        const uint4 *qp = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + oh * D);
        const float below = (small >> (__ffs(rows) - 1)) & 1u ? 24.f : 0.f;
        float o[PER], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = 0.f;
        const int end = a.tree_mask ? k1 : min(k1, hi);
        for (int j0 = max(k0, lo) & ~31; j0 < end; j0 += 32) {
            const int j = j0 + lane;
            bool seen = j >= k0 && j < k1 && j >= lo && j < hi;
            if (a.tree_mask && j >= max(base, k0) && j < k1)
                seen = (__ldg(a.tree_mask + (size_t)(t.q0 + tok) * a.mask_words + ((j - base) >> 5)) >>
                        ((j - base) & 31)) & 1u;
            size_t at = 0;
            if (seen) {
                const int b = __ldg(a.block_tables + (size_t)t.seq * a.max_blocks_per_seq + j / a.block_size);
                seen = b >= 0 && b < a.num_blocks;
                if (seen) at = (((size_t)b * a.num_kv_heads + kvh) * a.block_size + j % a.block_size) * D;
            }
            const uint32_t any = __ballot_sync(0xffffffffu, seen);
            if (any == 0) continue;
            float x = -CUDART_INF_F;
            if (seen) {
                const uint4 *kp = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.k_pool) + at);
                x = 0.f;
#pragma unroll 4
                for (int i = 0; i < D / kVec; ++i) {
                    const uint4 q = __ldg(qp + i), k = __ldg(kp + i);
                    const uint32_t qw[4] = {q.x, q.y, q.z, q.w}, kw[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x = fmaf(Mma16<T>::lo(qw[e]), Mma16<T>::lo(kw[e]), x);
                        x = fmaf(Mma16<T>::hi(qw[e]), Mma16<T>::hi(kw[e]), x);
                    }
                }
                x *= a.scale;
                if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                x = x * kTcLog2e - (a.slopes ? slope * fabsf((float)(pos - j)) : 0.f);
            }
            float top = fmaxf(m, x);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            const float f = exp2f(m - ref), p = seen ? exp2f(x - ref - below) : 0.f;
            m = top;
            l = l * f + p;  // (the lanes' sums are joined at the end)
#pragma unroll
            for (int i = 0; i < PER; ++i) o[i] *= f;
#pragma unroll 4
            for (int s = 0; s < 32; ++s) {
                const float w = __shfl_sync(0xffffffffu, p, s);
                const size_t from = __shfl_sync(0xffffffffu, at, s);
                if ((any >> s) & 1u) {
                    const T *vp = static_cast<const T *>(a.v_pool) + from;
#pragma unroll
                    for (int i = 0; i < PER; ++i) o[i] = fmaf(w, (float)vp[i * 32 + lane], o[i]);
                }
            }
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (a.num_parts > 1 && lane == 0)
            a.ws_lse[oh * a.num_parts + part] = l == 0.f ? -CUDART_INF_F : m + below + log2f(l);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (a.num_parts > 1)
                a.ws_o[(oh * a.num_parts + part) * D + i * 32 + lane] = o[i] * inv;
            else
                store_out(a.out, oh * D + i * 32 + lane, o[i] * inv, a.out_dtype);
        }
    }
}

// Uniform figures of capped and biased scores, in log2 units.
struct TcForm {
    float scale;            // of a score
    float cap, in_e;        // softcap; x = scale q.k / cap: 2 x / q.k in log2 units
    float small;            // |q.k| up to which |x| <= 0.3: the polynomial's range
    float c1, c3, c5, c7;   // cap tanh(x) = v (c1 + c3 v^2 + c5 v^4 + c7 v^6) with v = q.k, |x| <= 0.3
    bool capped, biased, both_ways;
};

__device__ __forceinline__ TcForm tc_form(const ExtArgs &a) {
    TcForm f;
    f.scale = fabsf(a.scale) * kTcLog2e;
    f.capped = a.softcap > 0.f, f.biased = a.slopes != nullptr, f.both_ways = a.prefix_lens != nullptr;
    f.cap = a.softcap * kTcLog2e;
    const float in = f.capped ? fabsf(a.scale) / a.softcap : 0.f;
    f.in_e = 2.f * kTcLog2e * in;
    // (of larger `in` the coefficients may overflow, of larger q.k their square)
    f.small = in <= 1e4f ? fminf(0.3f / in, 1e19f) : -1.f;
    // tanh(x) / x as a polynomial in x^2, fitted on |x| <= 0.3: off by 4.3e-8 at most
    const float q = in * in;
    f.c1 = f.scale, f.c3 = -0.333332865f * f.scale * q, f.c5 = 0.133239105f * f.scale * q * q,
    f.c7 = -0.0511367784f * f.scale * q * q * q;
    return f;
}

// W scores q.k (of a row, for adjacent keys) capped and biased, in log2 units;
// they are in s, and in TMEM from column `col` on, where they may be overwritten.
// `dist`: the row's position less the first key's.
//
// A score's cap is a function of that score alone: the polynomial up to `small`,
// above it cap (1 - 2 / (1 + e^(2 x))), whose error of some 2^-22 of the cap a
// small score would not bear.  Other scores of the warp, among them those of
// keys that a row does not see, decide only whether the second form is computed
// at all.
template <int W>
__device__ __forceinline__ void tc_modify(float *s, uint32_t col, const TcForm &f, float slope, int dist) {
    if (f.capped) {
        float big = 0.f, also = 0.f;
#pragma unroll
        for (int e = 0; e < W; e += 4) {
            big = max3(big, fabsf(s[e]), fabsf(s[e + 1]));
            also = max3(also, fabsf(s[e + 2]), fabsf(s[e + 3]));
        }
        big = fmaxf(big, also);
        if (__all_sync(0xffffffffu, big <= f.small)) {
            // the FMA pipe has room where the exponential and the reciprocal of
            // the other form would fill theirs
            const F2 c1 = f2_pack(f.c1, f.c1), c3 = f2_pack(f.c3, f.c3), c5 = f2_pack(f.c5, f.c5),
                     c7 = f2_pack(f.c7, f.c7);
#pragma unroll
            for (int e = 0; e < W; e += 2) {
                const F2 v = f2_pack(s[e], s[e + 1]), t = f2_mul(v, v);
                f2_unpack(f2_mul(v, f2_fma(t, f2_fma(t, f2_fma(t, c7, c5), c3), c1)), s[e], s[e + 1]);
            }
        } else {
            // The polynomial by single operations, which round alike, in a loop over
            // the scores in TMEM.  Laid out W times, this code made the other branch
            // slower (mixed step 179.7 -> 184.2 us) and took longer itself (8 chunks
            // of 700 tokens over 2300, head_dim 128, cap 5: 396 -> 440), as packed
            // operations did, whose constants stay in registers (183.9, 414).
#pragma unroll 1
            for (int n = 0; n < W; n += 16) {
                float u[16];
                tmem_ld16_now(col + n, u);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float v = u[e], t = v * v;
                    const float near = v * fmaf(t, fmaf(t, fmaf(t, f.c7, f.c5), f.c3), f.c1);
                    const float far = fmaf(-2.f * f.cap, fast_rcp(1.f + fast_exp2(v * f.in_e)), f.cap);
                    u[e] = fabsf(v) <= f.small ? near : far;
                }
                tmem_st16(col + n, u);
            }
            tmem_wait_st();
#pragma unroll
            for (int n = 0; n < W; n += 32) tmem_ld32(col + n, s + n);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < W; n += 32) tmem_pin32(s + n);
        }
    }
    if (f.biased) {
        // -slope (dist - e) = slope e - slope dist: two roundings of the bias
        const float unit = f.capped ? 1.f : f.scale, base = -slope * (float)dist;
        if (f.both_ways && __any_sync(0xffffffffu, dist < W - 1)) {
            // keys behind the row, which are seen only where there is a prefix
#pragma unroll
            for (int e = 0; e < W; ++e) s[e] = fmaf(s[e], unit, -slope * fabsf((float)(dist - e)));
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) s[e] = fmaf(s[e], unit, fmaf(slope, (float)e, base));
        }
    }
}

// Weights 2^(s factor + shift) of 32 scores, written to TMEM columns col ..
// col + 31 as A operands of P V, and added to the sums: in the pool's type, two
// to a column, at col.  Where the output has 16 bits that rounding is no
// larger than its own.  Where it has 32 (SPLIT), the weights' remainders
// follow at col + 16 as a second operand.
template <typename T, bool SPLIT>
__device__ __forceinline__ void tc_weights(float *s, uint32_t col, F2 f2, F2 h2, F2 &sum0, F2 &sum1) {
#pragma unroll
    for (int i = 0; i < 32; i += 16) {
        uint32_t ph[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float &x = s[i + 2 * e], &y = s[i + 2 * e + 1];
            f2_unpack(f2_fma(f2_pack(x, y), f2, h2), x, y);
            x = fast_exp2(x), y = fast_exp2(y);
            (e & 1 ? sum1 : sum0) = f2_add(e & 1 ? sum1 : sum0, f2_pack(x, y));
            ph[e] = Mma16<T>::pack(x, y);
        }
        tmem_st8(col + i / 2, ph);
        if constexpr (SPLIT) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                ph[e] = Mma16<T>::pack(s[i + 2 * e] - Mma16<T>::lo(ph[e]),
                                       s[i + 2 * e + 1] - Mma16<T>::hi(ph[e]));
            tmem_st8(col + 16 + i / 2, ph);
        }
    }
}

// CTA: NQ tiles of 128 rows, one kv head, one part of its keys.
template <typename T, int D, int NQ, bool MODS, bool SPLIT>
__global__ void __launch_bounds__(TcShape<D, NQ>::kThreads, TcShape<D, NQ>::kCtas)
    extend_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const ExtArgs a) {
    using S = TcShape<D, NQ>;
    constexpr int KT = S::KT, NS = S::NS, NK = S::NK, NV = S::NV, RUNS = KT / kExtRun;
    constexpr int kLoadWarp = NQ * 4, kMmaWarp = kLoadWarp + 1;
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *qs = sm, *ring = sm + NQ * S::kQBytes;
    TcControl &c = *reinterpret_cast<TcControl *>(sm + S::kTiles);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    griddep_wait();
    ext_check_starts(a);
    const int kvh = blockIdx.x % a.num_kv_heads;
    // side by side: the CTA's item is found, barriers and TMEM are set up
    if (warp == 0) {
        ExtTile t;
        int part, k0 = 0, k1 = 0;
        if (!ext_find_item(a, blockIdx.x / a.num_kv_heads, S::kRows, t, part)) part = -1;
        if (part >= 0) ext_part(a, t, part, k0, k1);
        if (lane == 0) {
            c.tile = t, c.part = part;
            c.k0 = k0, c.k1 = k1;
        }
        if (lane == 0 && k0 < k1) {
            const int active = (t.nrows + 31) / 32;
            const int nq = NQ == 2 && t.nrows > 128 ? 2 : 1;  // row tiles with rows
            for (int i = 0; i < NK + NV; ++i) mbar_init(&c.empty[i], nq);
            for (int i = 0; i < 2; ++i) {
                const int sets = min(4, max(1, NQ == 2 ? active - 4 * i : active));
                mbar_init(&c.p_half[i], sets), mbar_init(&c.p_ready[i], sets);
            }
            c.base = t.ctx - t.ntok;
            c.ntok = t.ntok, c.q0 = t.q0, c.prefix = t.prefix;
            // rows are in token order: the first sees the fewest keys at the end,
            // the last the fewest at the start
            const int first_pos = c.base + t.row0 / a.group, last_pos = c.base + (t.row0 + t.nrows - 1) / a.group;
            int dump;
            c.kmin = 0, c.same_lo = 0, c.same_hi = c.base;
            if (!a.tree_mask) {
                ext_row_range(a, t.prefix, first_pos, c.kmin, c.same_hi);
                ext_row_range(a, t.prefix, last_pos, c.same_lo, dump);
            }
            c.inner_lo = max(c.kmin, c.same_lo), c.inner_hi = min(k1, c.same_hi);
            fence_mbar_init();
        }
    } else if (warp == 1 && lane == 0) {
        for (int i = 0; i < NK + NV; ++i) mbar_init(&c.full[i], 1);
        for (int i = 0; i < 2; ++i) {  // by row tile, or by score tile where there is one row tile
            mbar_init(&c.s_full[i], 2);
            mbar_init(&c.o_full[i], 1);
            mbar_init(&c.o_last[i], 1);
            mbar_init(&c.turn[i], 1);
        }
        mbar_init(&c.q_full, kLoadWarp * 32);
        c.stop = 0;
        fence_mbar_init();
    } else if (warp == kMmaWarp) {
        // after griddep_wait: no earlier grid of the stream can hold TMEM while it
        // waits for this one
        tmem_alloc(&c.tmem, S::kCols);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch();
    const ExtTile t = c.tile;
    const int part = c.part, k0 = c.k0, k1 = c.k1;
    const int ntiles = (k1 - k0 + KT - 1) / KT;
    const int G = a.group;
    const int active = (t.nrows + 31) / 32;  // sets of 32 rows

    if (part < 0 || ntiles == 0) {  // no item, or nothing to see
        for (int r = warp; part >= 0 && r < t.nrows; r += S::kThreads / 32) {
            const int row = t.row0 + r, tok = row / G;
            const size_t oh = (size_t)(t.q0 + tok) * a.num_heads + kvh * G + row - tok * G;
            if (a.num_parts > 1) {
                if (lane == 0) a.ws_lse[oh * a.num_parts + part] = -CUDART_INF_F;
            } else {
                for (int d = lane; d < D; d += 32) store_out(a.out, oh * D + d, 0.f, a.out_dtype);
            }
        }
        if (warp == kMmaWarp) tmem_free(c.tmem, S::kCols);
        return;
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);

    if (warp < kLoadWarp) {
        // queries, in the 128-byte swizzle the products read; the softmax warps'
        // rows behind the last are zero, so that no time or result depends on what
        // the memory held
        constexpr int C = D / 8, kStep = kLoadWarp * 32 / C;
        const int ch = tid % C, step_tok = kStep / G, step_g = kStep % G;
        int tok = (t.row0 + tid / C) / G, g = t.row0 + tid / C - tok * G;
        int r = tid / C;
#pragma unroll 2
        for (; r < t.nrows; r += kStep) {
            const uint32_t dst = smem_u32(qs) + (r / 128) * S::kQBytes + swz_offset<128>(r % 128, ch);
            const void *src = static_cast<const T *>(a.q) +
                              ((size_t)(t.q0 + tok) * a.num_heads + kvh * G + g) * D + ch * 8;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
            tok += step_tok, g += step_g;
            if (g >= G) g -= G, ++tok;
        }
        for (; r < active * 32; r += kStep) sts_zero16(smem_u32(qs) + (r / 128) * S::kQBytes + swz_offset<128>(r % 128, ch));
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (a.scale < 0.f) {  // the products take |scale|
            for (r = tid / C; r < t.nrows; r += kStep) {
                uint4 *p = reinterpret_cast<uint4 *>(qs + (r / 128) * S::kQBytes + swz_offset<128>(r % 128, ch));
                uint4 v = *p;
                v.x ^= 0x80008000u, v.y ^= 0x80008000u, v.z ^= 0x80008000u, v.w ^= 0x80008000u;
                *p = v;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(&c.q_full);
    }
    if (warp == kLoadWarp) {
        // ------------------------------------------------- staging of K and V
        const uint64_t policy = l2_evict_first_policy();
        const int32_t *tbl = a.block_tables + (size_t)t.seq * a.max_blocks_per_seq;
        const int run0 = k0 / kExtRun, run_end = (k1 + kExtRun - 1) / kExtRun;
        const int run_min = c.kmin / kExtRun;
        auto block_of = [&](int run) {
            return run >= run_min && run < run_end ? __ldg(tbl + (run >> a.run_shift)) : -1;
        };
        // tiles are taken from the last, whose keys are nearest to the rows: a
        // distance bias then leaves the largest scores to the first tile.  A lane
        // holds the block number of one of 32 runs, and of one of the 32 before.
        constexpr int kPer = 32 / RUNS;
        int now = 0, next = block_of(run0 + (ntiles - 1) / kPer * 32 + lane);
        bool ok = true;
        // One tile of K or V.  One thread issues all copies: lanes that each issue
        // their own take turns at it, and longer.
        auto stage = [&](const CUtensorMap &map, int buf, int use, uint32_t runs, const int (&ys)[RUNS]) {
            ok = ok && __all_sync(0xffffffffu, tc_wait(c, &c.empty[buf], (use & 1) ^ 1, a.dev_error));
            if (ok && elect_one()) {
                mbar_arrive_expect_tx(&c.full[buf], __popc(runs) * kExtRun * D * 2);
                unsigned char *dst = ring + buf * S::kTileBytes;
#pragma unroll
                for (int i = 0; i < RUNS; ++i)
                    if ((runs >> i) & 1u) {
#pragma unroll
                        for (int x = 0; x < S::kSlabs; ++x)
                            tma_load_2d_hint(dst + i * (kExtRun * 128) + x * (KT * 128), &map, x * 64,
                                             ys[i], &c.full[buf], policy);
                    }
            }
            __syncwarp();
        };
        // Where two score tiles let the next tile's products run ahead, its K is
        // wanted before this one's V.
        constexpr int kLag = NS - 1;
        uint32_t v_mask = 0;
        int v_ys[RUNS];
        for (int j = 0; j < ntiles && ok; ++j) {
            const int tile = ntiles - 1 - j;
            if (j == 0 || tile % kPer == kPer - 1) {
                now = next;
                next = tile >= kPer ? block_of(run0 + (tile / kPer - 1) * 32 + lane) : -1;
            }
            const int r = lane % RUNS, run = run0 + tile * RUNS + r;
            const int blk = __shfl_sync(0xffffffffu, now, (tile % kPer) * RUNS + r);
            const bool wanted = run >= run_min && run < run_end;
            const bool valid = wanted && blk >= 0 && blk < a.num_blocks;
            if (wanted && !valid && lane < RUNS) raise_fault(a.dev_error, PKV_FAULT_BLOCK_ID);
            const uint32_t mask = __ballot_sync(0xffffffffu, valid) & ((1u << RUNS) - 1u);
            const int y = (int)((((long long)blk * a.num_kv_heads + kvh) << a.run_shift) * kExtRun) +
                          (run & ((1 << a.run_shift) - 1)) * kExtRun;
            int ys[RUNS];
#pragma unroll
            for (int i = 0; i < RUNS; ++i) ys[i] = __shfl_sync(0xffffffffu, y, i);
            if (lane == 0) c.bad[j & 7] = ~mask;
            __syncwarp();
            stage(tmk, j % NK, j / NK, mask, ys);
            if (j >= kLag) stage(tmv, NK + (j - kLag) % NV, (j - kLag) / NV, kLag ? v_mask : mask, kLag ? v_ys : ys);
            v_mask = mask;
#pragma unroll
            for (int i = 0; i < RUNS; ++i) v_ys[i] = ys[i];
        }
        if (kLag) stage(tmv, NK + (ntiles - 1) % NV, (ntiles - 1) / NV, v_mask, v_ys);
        if (c.stop) {  // given up: wait for the copies in flight before the memory goes
            for (int i = 0; i < NK + NV; ++i) mbar_wait_for(&c.full[i], 0, 1000000ull), mbar_wait_for(&c.full[i], 1, 1000000ull);
        }
    } else if (warp >= kMmaWarp) {
        // ---------------------------------------------------------- products
        // A warp per row tile: it runs the loop together and one elected thread
        // issues.  The loops over k are not unrolled: a product takes 64 cycles,
        // far longer than its issue, and short code stays in the instruction
        // cache beside the softmax's.
        constexpr uint32_t id_s = mma_idesc(kBf16, false, 128, KT);
        constexpr uint32_t id_o = mma_idesc(kBf16, true, 128, D);
        const int q = warp - kMmaWarp;
        const uint32_t ring_at = smem_u32(ring), o = tmem + S::kOCol + q * D;
        const uint64_t dq = smem_desc(smem_u32(qs + q * S::kQBytes), 16, 1024);
        bool ok = q * 128 < t.nrows;
        const bool two = NQ == 2 && t.nrows > 128;
        auto wait = [&](uint64_t *bar, unsigned parity) {
            ok = ok && __all_sync(0xffffffffu, tc_wait(c, bar, parity, a.dev_error));
        };
        // products of one tile, issued by the elected thread
        auto scores = [&](int j) {
            const int buf = j % NK, at = NQ == 2 ? q : j % NS;
            const uint64_t dk = smem_desc(ring_at + buf * S::kTileBytes, 16, 1024);
            mbar_arrive(&c.s_full[at]);  // carries the staging warp's writes to the readers
#pragma unroll 1
            for (int s = 0; s < S::kSlabs; ++s)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss(tmem + at * KT, dq + (s * (128 * 128) + k * 32) / 16,
                           dk + (s * (KT * 128) + k * 32) / 16, id_s, s > 0 || k > 0);
            mma_commit(&c.s_full[at]);
            mma_commit(&c.empty[buf]);
        };
        auto output = [&](int j, int k_begin, int k_end) {
            const int buf = NK + j % NV;
            const uint64_t dv = smem_desc(ring_at + buf * S::kTileBytes, KT * 128, 1024);
            const uint32_t p = tmem + (NQ == 2 ? q : j % NS) * KT;
#pragma unroll 1
            for (int k = k_begin; k < k_end; ++k) {
                mma_ts(o, p + k * 32, dv + k * (32 * 128) / 16, id_o, j > 0 || k > 0);
                mma_ts(o, p + k * 32 + 8, dv + (k * 32 + 16) * 128 / 16, id_o, true);
                if constexpr (SPLIT) {
                    mma_ts(o, p + k * 32 + 16, dv + k * (32 * 128) / 16, id_o, true);
                    mma_ts(o, p + k * 32 + 24, dv + (k * 32 + 16) * 128 / 16, id_o, true);
                }
            }
        };
        auto output_done = [&](int j) {
            mma_commit(&c.empty[NK + j % NV]);
            mma_commit(&c.o_full[q]);
            if (j + 1 == ntiles) mma_commit(&c.o_last[q]);
        };
        auto wait_k = [&](int j) { wait(&c.full[j % NK], (j / NK) & 1); };
        auto wait_v = [&](int j) { wait(&c.full[NK + j % NV], (j / NV) & 1); };
        // The products of a thread run in the order of their issue: a score
        // tile that overwrites weights follows the product that reads them.
        wait(&c.q_full, 0);
        wait_k(0);
        tc_fence_after();
        if (ok && elect_one()) scores(0);
        __syncwarp();
        for (int j = 0; j < ntiles && ok; ++j) {
            const bool more = j + 1 < ntiles;
            if (NS > 1 && more) {
                wait_k(j + 1);
                tc_fence_after();
                if (ok && elect_one()) scores(j + 1);
                __syncwarp();
            }
            wait_v(j);
            if (NQ == 2 && more) wait_k(j + 1);
            // Two row tiles take turns: while one's products run, the other is
            // in softmax.  (Row tile 0's turn also comes after its softmax has
            // cleared the rows of V that no row sees.)
            if (two) wait(&c.turn[1 - q], q ? j & 1 : (j & 1) ^ 1);
            if (NQ == 2) {  // the first half's product runs beside the other half's softmax
                wait(&c.p_half[q], j & 1);
                tc_fence_after();
                if (ok && elect_one()) output(j, 0, KT / 64);
                __syncwarp();
            }
            wait(&c.p_ready[NQ == 2 ? q : j % NS], (j / NS) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                output(j, NQ == 2 ? KT / 64 : 0, KT / 32);
                output_done(j);
                if (NQ == 2 && more) scores(j + 1);
                if (two) mbar_arrive(&c.turn[q]);
            }
            __syncwarp();
        }
        if (!ok && q * 128 < t.nrows) {  // given up: the products issued must end before TMEM goes
            if (elect_one()) mma_commit(&c.o_full[q]);
            mbar_wait_for(&c.o_full[q], 0, 1000000ull), mbar_wait_for(&c.o_full[q], 1, 1000000ull);
            __syncwarp();
        }
    } else if (warp < active) {
        // ----------------------------------------------------------- softmax
        const int q = warp / 4;
        const uint32_t lanes = tmem + ((uint32_t)(warp % 4) << 21);
        const uint32_t ocol = lanes + S::kOCol + q * D;
        const int r = warp * 32 + lane;
        const bool live = r < t.nrows;
        const int row = t.row0 + (live ? r : t.nrows - 1), tok = row / G, h = kvh * G + row - tok * G;
        const int pos = c.base + tok;
        const int inner_lo = c.inner_lo, inner_hi = c.inner_hi;
        const float slope = MODS && a.slopes ? __ldg(a.slopes + h) * kTcLog2e : 0.f;
        const TcForm form = tc_form(a);
        // scores in log2 units; a scale of zero stays above it, so that -inf * factor is -inf
        const float factor = MODS ? 1.f : fmaxf(fabsf(a.scale) * kTcLog2e, 1e-30f);
        // l is zero until the row has seen a key.
        using Ref = TcRef<kBf16>;
        float m = 0.f, l = 0.f;
        bool ok = true;
        for (int j = 0; j < ntiles; ++j) {
            const int k = k0 + (ntiles - 1 - j) * KT;
            const int at = NQ == 2 ? q : j % NS;
            ok = __all_sync(0xffffffffu, tc_wait(c, &c.s_full[at], (j / NS) & 1, a.dev_error));
            if (!ok) break;
            tc_fence_after();
            const uint32_t scol = lanes + at * KT;
            const uint32_t bad = c.bad[j & 7];
            // every row sees the whole tile
            const bool whole = k >= inner_lo && k + KT <= inner_hi && (bad & ((1u << RUNS) - 1u)) == 0;
            // The scores' maximum.  A tile of 64 keys stays in registers until its
            // weights are written; one of 128 is read again, and written back where
            // it is masked.  The loops over a tile stay rolled: unrolled, the code
            // did not fit the instruction caches and its misses took longer than
            // the arithmetic.
            constexpr bool kHeld = KT == 64;
            static_assert(kHeld || !MODS, "modified scores are held");
            float t0 = -CUDART_INF_F, t1 = t0, s[64];
            // what the row sees, within the part
            int lo = 0, hi = c.base;
            const uint32_t *words = nullptr;
            if (!whole) {
                if (a.tree_mask) words = a.tree_mask + (size_t)(c.q0 + pos - c.base) * a.mask_words;
                else ext_row_range(a, c.prefix, pos, lo, hi);
                hi = min(hi, c.k1);
            }
            auto scan = [&](auto masked) {
#pragma unroll 1
                for (int n = 0; n < KT; n += 64) {
                    tmem_ld32(scol + n, s), tmem_ld32(scol + n + 32, s + 32);
                    tmem_wait_ld();
                    tmem_pin32(s), tmem_pin32(s + 32);
                    if constexpr (MODS) tc_modify<64>(s, scol + n, form, slope, pos - k);
                    if (masked()) {
#pragma unroll
                        for (int i = 0; i < 64; i += 32) {
                            const uint32_t see = tc_seen(a, c, lo, hi, words, k, (n + i) / 32, bad);
                            if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!((see >> e) & 1u)) s[i + e] = -CUDART_INF_F;
                                if (!kHeld) tmem_st32(scol + n + i, s + i);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 64; e += 4)
                        t0 = max3(t0, s[e], s[e + 1]), t1 = max3(t1, s[e + 2], s[e + 3]);
                }
                if (!kHeld) tmem_wait_st();
            };
            if constexpr (kHeld) {
                scan([&] { return !whole; });
            } else if (whole) {
                scan([] { return false; });
            } else {
                scan([] { return true; });
            }
            const float top = fmaxf(t0, t1) * factor;
            const bool move = l == 0.f ? top > -CUDART_INF_F : top > m + Ref::kLag;
            if (__any_sync(0xffffffffu, move)) {
                const bool scale_o = move && l != 0.f;
                if (__any_sync(0xffffffffu, scale_o)) {
                    // O must hold the products up to the last tile's, and no later one
                    ok = __all_sync(0xffffffffu, tc_wait(c, &c.o_full[q], (j - 1) & 1, a.dev_error));
                    if (!ok) break;
                    tc_fence_after();
                    const float f = scale_o ? fast_exp2(m - (top - Ref::kBelow)) : 1.f;
                    l *= f;
#pragma unroll 1
                    for (int i = 0; i < D / 16; ++i) {
                        float o[16];
                        tmem_ld16_now(ocol + i * 16, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= f;
                        tmem_st16(ocol + i * 16, o);
                    }
                }
                if (move) m = top - Ref::kBelow;
            }
            const F2 f2 = f2_pack(factor, factor), h2 = f2_pack(-m, -m);
            F2 sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll 1
            for (int n = 0; n < KT; n += 64) {
                if (!kHeld) {
                    tmem_ld32(scol + n, s), tmem_ld32(scol + n + 32, s + 32);
                    tmem_wait_ld();
                    tmem_pin32(s), tmem_pin32(s + 32);
                }
                tc_weights<T, SPLIT>(s, scol + n, f2, h2, sum0, sum1);
                tc_weights<T, SPLIT>(s + 32, scol + n + 32, f2, h2, sum0, sum1);
                if (NQ == 2 && n == 0 && whole) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.p_half[q]);
                }
            }
            float sum_x, sum_y;
            f2_unpack(f2_add(sum0, sum1), sum_x, sum_y);
            l += sum_x + sum_y;
            if (q == 0 && !whole) {
                const int lo = max(c.kmin - k, 0), hi = min(c.k1 - k, KT);
                // runs that no row sees, of those that are not before or behind all
                uint32_t gone = bad & ((1u << RUNS) - 1u) & (0xffffffffu << (lo / kExtRun));
                gone &= (1u << ((hi + kExtRun - 1) / kExtRun)) - 1u;
                if (lo > 0 || hi < KT || gone) {
                    const int buf = NK + j % NV, warps = min(active, 4);
                    ok = __all_sync(0xffffffffu, tc_wait(c, &c.full[buf], (j / NV) & 1, a.dev_error));
                    if (!ok) break;
                    tc_clear_values<D, KT>(ring + buf * S::kTileBytes, lo, hi, gone, tid, warps * 32);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (NQ == 2 && !whole) mbar_arrive(&c.p_half[q]);  // not before V is cleared
                mbar_arrive(&c.p_ready[at]);
            }
        }
        // ------------------------------------------------------------ result
        // (a barrier of its own: a wait on o_full may be two phases behind here,
        // and a parity tells only one)
        ok = ok && __all_sync(0xffffffffu, tc_wait(c, &c.o_last[q], 0, a.dev_error));
        if (ok) {
            tc_fence_after();
            const bool split = a.num_parts > 1;
            const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN where a visible score was
            if (split && live)
                a.ws_lse[((size_t)(c.q0 + tok) * a.num_heads + h) * a.num_parts + part] =
                    l == 0.f ? -CUDART_INF_F : m + log2f(l);
            // The warp's rows go through the queries' shared memory (no product
            // reads it any more), so that whole rows are written at once.
            const int type = split ? PKV_F32 : a.out_dtype;
            const int row_bytes = type == PKV_F32 ? 4 * D : 2 * D;
            unsigned char *stage = qs + warp * (32 * 2 * D);  // 32 rows of 2 D bytes
            constexpr int C = 2 * D / 16;                     // chunks of a staged row
            const int nlive = min(32, t.nrows - warp * 32);
            bool nan = false, odd = false;
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += type == PKV_F32 ? D / 2 : D) {
                __syncwarp();
#pragma unroll 1
                for (int x = 0; x < (type == PKV_F32 ? D / 2 : D); x += 32) {
                    float v[32];
                    tmem_ld32(ocol + d0 + x, v);
                    tmem_wait_ld();
                    tmem_pin32(v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] *= inv;
                        nan |= v[e] != v[e];
                        odd |= !(fabsf(v[e]) <= 3e38f);
                    }
                    uint4 *dst = reinterpret_cast<uint4 *>(stage + lane * (2 * D));
                    if (type == PKV_F32) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[(x / 4 + e) ^ (lane & 7)] =
                                make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]),
                                           __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[i] = type == PKV_BF16 ? pack_bf16(v[8 * e + 2 * i], v[8 * e + 2 * i + 1])
                                                        : pack_f16(v[8 * e + 2 * i], v[8 * e + 2 * i + 1]);
                            dst[(x / 8 + e) ^ (lane & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                __syncwarp();
                constexpr int kStep = 32 / C > 0 ? 32 / C : 1;  // rows of an iteration
                const int first = t.row0 + warp * 32 + (C < 32 ? lane / C : 0);
                const int step_tok = kStep / G, step_g = kStep % G;
                int otok = first / G, og = first - otok * G;
#pragma unroll 4
                for (int rr = C < 32 ? lane / C : 0; rr < nlive; rr += kStep) {
                    const size_t oh = (size_t)(c.q0 + otok) * a.num_heads + kvh * G + og;
                    char *base = split ? reinterpret_cast<char *>(a.ws_o) +
                                             (oh * a.num_parts + part) * row_bytes
                                       : static_cast<char *>(a.out) + oh * row_bytes;
                    const int ch = lane % C;
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        stage + rr * (2 * D) + ((ch ^ (rr & 7)) << 4));
                    *reinterpret_cast<uint4 *>(base + d0 * 4 * (type == PKV_F32) + ch * 16) = v;
                    otok += step_tok, og += step_g;
                    if (og >= G) og -= G, ++otok;
                }
            }
            odd = odd && live && l == l;
            if (__any_sync(0xffffffffu, odd)) {
                int lo = 0, hi = c.base;
                const uint32_t *words = nullptr;
                if (a.tree_mask) words = a.tree_mask + (size_t)(c.q0 + tok) * a.mask_words;
                else ext_row_range(a, c.prefix, pos, lo, hi);
                const int how = tc_not_its_own<T, D>(a, c, t.seq, kvh, odd && nan, odd && !nan, lo, hi, words);
                const uint32_t again = __ballot_sync(0xffffffffu, how != 0);
                const uint32_t small = __ballot_sync(0xffffffffu, how == 2);
                if (again) {
                    __syncwarp();
                    tc_redo_rows<T, D>(a, t, kvh, k0, k1, part, warp * 32, again, small);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, S::kCols);
}

template <typename T, int D, int NQ, bool MODS, bool SPLIT>
pkv_status launch_tc_one(const ExtLaunch &L) {
    using S = TcShape<D, NQ>;
    auto kern = extend_tc_kernel<T, D, NQ, MODS, SPLIT>;
    constexpr int smem = S::kTiles + (int)sizeof(TcControl);
    static_assert(smem <= 227 * 1024, "shared memory budget");
    static_assert(S::kCtas * (smem + 1024) <= 228 * 1024, "CTAs per SM");
    static unsigned long long done_mask = 0ull;
    const unsigned long long bit = 1ull << (L.device & 63);
    if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem)) != PKV_OK)
            return PKV_ERR_CUDA;
        __atomic_fetch_or(&done_mask, bit, __ATOMIC_RELEASE);
    }
    const dim3 grid((unsigned)L.args.tiles * L.args.num_kv_heads * L.args.num_parts);
    return cuda_status(launch_dependent(kern, grid, dim3(S::kThreads), smem, L.stream, *L.tmk,
                                        *L.tmv, L.args));
}

template <typename T, int D>
pkv_status launch_tc(const ExtLaunch &L) {
    const bool split = L.args.out_dtype == PKV_F32;
    if constexpr (D == 128)  // (scores are as they are)
        if (L.rows == 256)
            return split ? launch_tc_one<T, D, 2, false, true>(L) : launch_tc_one<T, D, 2, false, false>(L);
    if (L.args.softcap > 0.f || L.args.slopes)
        return split ? launch_tc_one<T, D, 1, true, true>(L) : launch_tc_one<T, D, 1, true, false>(L);
    return split ? launch_tc_one<T, D, 1, false, true>(L) : launch_tc_one<T, D, 1, false, false>(L);
}

}  // namespace pkv
