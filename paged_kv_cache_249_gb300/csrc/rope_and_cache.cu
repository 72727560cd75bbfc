// rope_and_cache.cu -- the cache write of a rotary model's new tokens in one
// pass: queries and keys are normalised per head (on request) and rotated by
// their position, queries go to their own buffer, keys and values to the
// paged cache.
//
// For a head's row x of D values, with w the norm's weight and (c_i, s_i) the
// cosine and sine of the token's position at frequency i < R/2:
//   x <- x * rsqrt(mean(x^2) + eps) * w                     (only with a weight)
//   y_a = x_a c_i - x_b s_i,  y_b = x_b c_i + x_a s_i
// where (a, b) is (i, i + R/2) in halves order and (2i, 2i + 1) in pairs
// order; values from R on pass.  Everything is fp32 and rounded once, to the
// pool's type, when the row is stored.
//
// Bound by HBM: every value is read and written once.  8192 tokens of 32 + 2 x 8
// heads of 128 in bf16 with both norms take 37 us (5.55 TB/s), 64 tokens 1.8 us.
#include <cmath>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kRopeThreads = 128;

struct RopeArgs {
    const void *query, *key, *value;  // [T] token rows of [heads][D], strides in bytes
    long long q_stride, k_stride, v_stride;
    void *query_out;                  // [T][H][D]
    void *k_pool, *v_pool;
    const int64_t *slot_mapping;
    const int32_t *positions;
    const float *cos_sin;             // [max_position][R]: R/2 cosines, then R/2 sines
    const void *q_norm, *k_norm;      // [D] in the pool's type, or NULL
    int32_t *dev_error;
    long long num_slots;
    float eps;
    int num_q_heads;                  // 0: no queries
    int num_kv_heads;
    int block_shift;                  // a block is 2^block_shift tokens
    int max_position;
    int rotary_dim;
};

// 16 bytes of T as floats, and back (one rounding to nearest even).
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
    static constexpr int V = 4;
    static __device__ __forceinline__ void load(const uint4 &r, float (&f)[4]) {
        f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <typename T>
struct Chunk16 {
    static constexpr int V = 8;
    static __device__ __forceinline__ void load(const uint4 &r, float (&f)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = Mma16<T>::lo(w[i]), f[2 * i + 1] = Mma16<T>::hi(w[i]);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(Mma16<T>::pack(f[0], f[1]), Mma16<T>::pack(f[2], f[3]),
                          Mma16<T>::pack(f[4], f[5]), Mma16<T>::pack(f[6], f[7]));
    }
};
template <>
struct Chunk<__nv_bfloat16> : Chunk16<__nv_bfloat16> {};
template <>
struct Chunk<__half> : Chunk16<__half> {};

template <int N>
__device__ __forceinline__ void load_floats(const float *p, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + i);
        f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
}

// Grid (token, set of rows): the rows of a token are its query, key and value
// heads.  A row is L = D*sizeof(T)/32 lanes; each lane owns two 16-byte chunks
// of it, chosen so that both members of every rotated pair are in one lane
// and no value crosses lanes: in halves order a chunk and the one R/2 further,
// in pairs order any two.  Only the norm's sum of squares is reduced over the
// L lanes.  A lane keeps its cosines and sines in registers for all its rows.
// As many CTAs share an SM as registers allow with hardly a spill: a row's loads,
// reduction and stores follow each other, and others' fill the gaps (8192 tokens
// with norms, three rows a thread: five CTAs 41.2 us, six 38.2, seven 37.0).
template <typename T, int D, int RPT, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, RPT == 4 ? 5 : RPT == 3 ? 7 : 8)
    rope_and_cache_kernel(const RopeArgs a) {
    using C = Chunk<T>;
    constexpr int V = C::V;
    constexpr int L = D / V / 2;              // lanes of a row
    constexpr int kRows = kRopeThreads / L;   // rows a pass of the CTA covers
    griddep_launch();
    griddep_wait();
    const int t = blockIdx.x;
    const int p = threadIdx.x % L, r0 = blockIdx.y * (kRows * RPT) + threadIdx.x / L;
    const int rows = a.num_q_heads + 2 * a.num_kv_heads;
    const int rot = a.rotary_dim;
    // the lane's two chunks
    int c0, c1;
    bool turn0, turn1;
    if (PAIRS) {
        c0 = p, c1 = p + L;
        turn0 = c0 * V < rot, turn1 = c1 * V < rot;
    } else {
        const int half = rot / (2 * V);  // chunks of half the rotated values
        if (p < half) {
            c0 = p, c1 = p + half;
        } else {
            c0 = p + half, c1 = c0 + (L - half);
        }
        turn0 = turn1 = p < half;
    }
    // the rows' values do not depend on slot or position, nor these on each
    // other: all are asked for at once
    const long long slot = __ldg(a.slot_mapping + t);
    const int pos = __ldg(a.positions + t);
    uint4 x0[RPT], x1[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + i * kRows;
        if (r < rows) {
            const char *src;
            if (r < a.num_q_heads)
                src = static_cast<const char *>(a.query) + t * a.q_stride + (size_t)r * D * sizeof(T);
            else if (r < a.num_q_heads + a.num_kv_heads)
                src = static_cast<const char *>(a.key) + t * a.k_stride +
                      (size_t)(r - a.num_q_heads) * D * sizeof(T);
            else
                src = static_cast<const char *>(a.value) + t * a.v_stride +
                      (size_t)(r - a.num_q_heads - a.num_kv_heads) * D * sizeof(T);
            x0[i] = *reinterpret_cast<const uint4 *>(src + c0 * 16);
            x1[i] = *reinterpret_cast<const uint4 *>(src + c1 * 16);
        } else {
            x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
        }
    }
    if (slot < 0) return;  // padding token: nothing of it is written
    if (slot >= a.num_slots || pos < 0 || pos >= a.max_position) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            raise_fault(a.dev_error, slot >= a.num_slots ? PKV_FAULT_SLOT : PKV_FAULT_POSITION);
        return;
    }
    // pairs order: a chunk's V values are V/2 pairs, cosines c0*V/2 and on for
    // the first chunk, c1*V/2 and on for the second; halves order: V cosines
    constexpr int N = PAIRS ? V / 2 : V;
    float cs0[N], sn0[N], cs1[PAIRS ? N : 1], sn1[PAIRS ? N : 1];
    const float *row = a.cos_sin + (size_t)pos * rot;
    if constexpr (PAIRS) {
        if constexpr (N >= 4) {
            if (turn0) load_floats<N>(row + c0 * N, cs0), load_floats<N>(row + rot / 2 + c0 * N, sn0);
            if (turn1) load_floats<N>(row + c1 * N, cs1), load_floats<N>(row + rot / 2 + c1 * N, sn1);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (turn0) cs0[i] = __ldg(row + c0 * N + i), sn0[i] = __ldg(row + rot / 2 + c0 * N + i);
                if (turn1) cs1[i] = __ldg(row + c1 * N + i), sn1[i] = __ldg(row + rot / 2 + c1 * N + i);
            }
        }
    } else if (turn0) {
        load_floats<N>(row + c0 * V, cs0), load_floats<N>(row + rot / 2 + c0 * V, sn0);
    }
    // (a pool has fewer than 2^31 rows)
    const int off = (int)slot & ((1 << a.block_shift) - 1), row0 = ((int)slot - off) * a.num_kv_heads + off;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + i * kRows;
        const bool is_q = r < a.num_q_heads;
        const int h = is_q ? r : r - a.num_q_heads;  // kv rows: keys, then values
        const bool is_v = !is_q && h >= a.num_kv_heads;
        const void *w = r < rows && !is_v ? (is_q ? a.q_norm : a.k_norm) : nullptr;
        float f0[V], f1[V];
        C::load(x0[i], f0);
        C::load(x1[i], f1);
        // the L lanes of a row agree on w, but the warp's rows may not: every
        // lane takes part in the reduction
        if (a.q_norm || a.k_norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(f0[e], f0[e], fmaf(f1[e], f1[e], ss));
#pragma unroll
            for (int m = L / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            if (w) {
                const float inv = rsqrtf(ss * (1.f / D) + a.eps);
                float w0[V], w1[V];
                C::load(__ldg(static_cast<const uint4 *>(w) + c0), w0);
                C::load(__ldg(static_cast<const uint4 *>(w) + c1), w1);
#pragma unroll
                for (int e = 0; e < V; ++e) f0[e] = f0[e] * inv * w0[e], f1[e] = f1[e] * inv * w1[e];
            }
        }
        if (r >= rows) continue;
        uint4 *dst;
        if (is_q)
            dst = reinterpret_cast<uint4 *>(static_cast<T *>(a.query_out) +
                                            ((size_t)t * a.num_q_heads + h) * D);
        else
            dst = reinterpret_cast<uint4 *>(
                static_cast<T *>(is_v ? a.v_pool : a.k_pool) +
                (size_t)(row0 + ((is_v ? h - a.num_kv_heads : h) << a.block_shift)) * D);
        if (is_v) {  // values are copied bit by bit
            dst[c0] = x0[i], dst[c1] = x1[i];
            continue;
        }
        if constexpr (PAIRS) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                if (turn0) {
                    const float u = f0[2 * e], v = f0[2 * e + 1];
                    f0[2 * e] = u * cs0[e] - v * sn0[e], f0[2 * e + 1] = v * cs0[e] + u * sn0[e];
                }
                if (turn1) {
                    const float u = f1[2 * e], v = f1[2 * e + 1];
                    f1[2 * e] = u * cs1[e] - v * sn1[e], f1[2 * e + 1] = v * cs1[e] + u * sn1[e];
                }
            }
        } else if (turn0) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = f0[e], v = f1[e];
                f0[e] = u * cs0[e] - v * sn0[e], f1[e] = v * cs0[e] + u * sn0[e];
            }
        }
        dst[c0] = C::pack(f0), dst[c1] = C::pack(f1);
    }
}

template <typename T, int D, bool PAIRS>
cudaError_t launch_rope_d(const RopeArgs &a, int num_tokens, cudaStream_t stream) {
    constexpr int kRows = kRopeThreads / (D / Chunk<T>::V / 2);
    const int rows = a.num_q_heads + 2 * a.num_kv_heads;
    auto launch = [&](auto kern, int rpt) {
        const dim3 grid((unsigned)num_tokens, (unsigned)((rows + kRows * rpt - 1) / (kRows * rpt)));
        return launch_dependent(kern, grid, dim3(kRopeThreads), 0, stream, a);
    };
    // With many tokens, as few CTAs for a token as hold its rows, up to four a
    // thread: cosines, sines and the token's slot serve more of them.  With few,
    // more CTAs: 64 tokens of 32 + 2 x 8 heads of 128 in bf16 take 1.8, 1.9, 2.1
    // and 2.2 us with 1 to 4 rows, 8192 tokens 38.5, 40.6, 36.7 and 37.1 (before
    // CTAs per SM were set; three hold the 48 rows).
    const int sets = (rows + kRows - 1) / kRows, ctas = (sets + 3) / 4;
    switch (num_tokens < 512 ? 1 : (sets + ctas - 1) / ctas) {
        case 1: return launch(rope_and_cache_kernel<T, D, 1, PAIRS>, 1);
        case 2: return launch(rope_and_cache_kernel<T, D, 2, PAIRS>, 2);
        case 3: return launch(rope_and_cache_kernel<T, D, 3, PAIRS>, 3);
        default: return launch(rope_and_cache_kernel<T, D, 4, PAIRS>, 4);
    }
}

template <typename T>
cudaError_t launch_rope(const RopeArgs &a, int head_dim, bool pairs, int num_tokens,
                        cudaStream_t stream) {
    if (pairs)
        return head_dim == 64    ? launch_rope_d<T, 64, true>(a, num_tokens, stream)
               : head_dim == 128 ? launch_rope_d<T, 128, true>(a, num_tokens, stream)
                                 : launch_rope_d<T, 256, true>(a, num_tokens, stream);
    return head_dim == 64    ? launch_rope_d<T, 64, false>(a, num_tokens, stream)
           : head_dim == 128 ? launch_rope_d<T, 128, false>(a, num_tokens, stream)
                             : launch_rope_d<T, 256, false>(a, num_tokens, stream);
}

// The angle position * frequency is formed and turned into cosine and sine in
// fp64: at position 10^5 an fp32 angle is off by up to 4e-3.  Run once per
// model, so its speed does not matter.
__global__ void __launch_bounds__(256)
    rope_table_kernel(float *cos_sin, const double *inv_freq, int half, long long total) {
    griddep_wait();
    const long long i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= total) return;
    const long long pos = i / half;
    const int f = (int)(i - pos * half);
    double s, c;
    sincos((double)pos * inv_freq[f], &s, &c);
    cos_sin[pos * 2 * half + f] = (float)c;
    cos_sin[pos * 2 * half + half + f] = (float)s;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_rope_table(float *cos_sin, int max_position, int rotary_dim, const double *inv_freq,
                          void *stream) {
    if (max_position <= 0 || rotary_dim <= 0 || rotary_dim % 16 != 0) return PKV_ERR_INVALID_ARG;
    if (rotary_dim > 256) return PKV_ERR_UNSUPPORTED;
    if (!cos_sin || !inv_freq || !aligned(cos_sin, 16) || !aligned(inv_freq, 8))
        return PKV_ERR_INVALID_ARG;
    const long long total = (long long)max_position * (rotary_dim / 2);
    if ((total + 255) / 256 > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent(rope_table_kernel, dim3((unsigned)((total + 255) / 256)),
                                        dim3(256), 0, static_cast<cudaStream_t>(stream), cos_sin,
                                        inv_freq, rotary_dim / 2, total));
}

pkv_status pkv_rope_and_cache(const pkv_pool *pool, void *query_out, const void *query,
                              int64_t query_stride, int num_heads, const void *key,
                              int64_t key_stride, const void *value, int64_t value_stride,
                              const int64_t *slot_mapping, const int32_t *positions,
                              const float *cos_sin, int max_position, int rotary_dim,
                              pkv_rope_order order, const void *query_norm, const void *key_norm,
                              float eps, int num_tokens, void *stream) {
    if (!pool || pool->magic != kPoolMagic || pool->layout != 0) return PKV_ERR_INVALID_ARG;
    if (num_tokens < 0 || num_heads < 0 || max_position <= 0) return PKV_ERR_INVALID_ARG;
    if (order != PKV_ROPE_HALVES && order != PKV_ROPE_PAIRS) return PKV_ERR_INVALID_ARG;
    if (rotary_dim <= 0 || rotary_dim > pool->head_dim || rotary_dim % 16 != 0)
        return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    const int elem = pool->dtype == PKV_F32 ? 4 : 2;
    const long long kv_row = (long long)pool->num_kv_heads * pool->head_dim;
    if ((num_heads > 0) != (query != nullptr) || (num_heads > 0) != (query_out != nullptr))
        return PKV_ERR_INVALID_ARG;
    if (num_heads == 0 && query_norm) return PKV_ERR_INVALID_ARG;
    if (!key || !value || !slot_mapping || !positions || !cos_sin) return PKV_ERR_INVALID_ARG;
    if (!aligned(query, 16) || !aligned(query_out, 16) || !aligned(key, 16) || !aligned(value, 16) ||
        !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(cos_sin, 16) ||
        !aligned(query_norm, 16) || !aligned(key_norm, 16))
        return PKV_ERR_INVALID_ARG;
    const long long q_row = (long long)num_heads * pool->head_dim;
    // token rows must not overlap, and start on 16 bytes
    if (key_stride < kv_row || value_stride < kv_row || (num_heads > 0 && query_stride < q_row))
        return PKV_ERR_INVALID_ARG;
    if ((key_stride * elem) % 16 != 0 || (value_stride * elem) % 16 != 0 ||
        (num_heads > 0 && (query_stride * elem) % 16 != 0))
        return PKV_ERR_INVALID_ARG;
    const long long limit = (1ll << 62) / num_tokens / elem;  // byte offsets stay in 64 bits
    if (key_stride > limit || value_stride > limit || (num_heads > 0 && query_stride > limit))
        return PKV_ERR_INVALID_ARG;
    // a row set per CTA in the grid's y
    if ((long long)num_heads + 2ll * pool->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != PKV_OK) return PKV_ERR_CUDA;
    if (dev != pool->device) return PKV_ERR_INVALID_ARG;
    RopeArgs a;
    a.query = query;
    a.key = key;
    a.value = value;
    a.q_stride = num_heads > 0 ? query_stride * elem : 0;
    a.k_stride = key_stride * elem;
    a.v_stride = value_stride * elem;
    a.query_out = query_out;
    a.k_pool = pool->k_pool;
    a.v_pool = pool->v_pool;
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.q_norm = query_norm;
    a.k_norm = key_norm;
    a.dev_error = pool->dev_error;
    a.num_slots = (long long)pool->num_blocks * pool->block_size;
    a.eps = eps;
    a.num_q_heads = num_heads;
    a.num_kv_heads = pool->num_kv_heads;
    a.block_shift = 0;
    while ((1 << a.block_shift) < pool->block_size) ++a.block_shift;
    a.max_position = max_position;
    a.rotary_dim = rotary_dim;
    const bool pairs = order == PKV_ROPE_PAIRS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int D = pool->head_dim;
    return cuda_status(pool->dtype == PKV_BF16  ? launch_rope<__nv_bfloat16>(a, D, pairs, num_tokens, st)
                       : pool->dtype == PKV_F16 ? launch_rope<__half>(a, D, pairs, num_tokens, st)
                                                : launch_rope<float>(a, D, pairs, num_tokens, st));
}

}  // extern "C"
