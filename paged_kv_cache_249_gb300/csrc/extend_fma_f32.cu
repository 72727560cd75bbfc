// extend_fma_f32.cu -- attention of several new tokens per sequence over fp32
// pools, on the CUDA cores in fp32 throughout.
//
// For a tile of query rows q_r (several tokens, all heads of one kv head) and
// the keys k_j, values v_j it sees:
//   s_rj = scale q_r.k_j,  capped, biased and masked;
//   m = max_j s_rj,  l = sum_j e^(s_rj - m),  out_r = sum_j e^(s_rj - m) v_j / l
// in one pass over the keys, with m and l running maxima and sums (in log2
// units) and the output rescaled when m grows.
//
// Bound: a tile needs R x 2 D multiply-adds for a key, of which an SM does 128
// a clock.  A thread's tile is 8 rows by 3 or 4 keys, then by D/16 columns: 11
// or 12 loads of 512 bytes a warp, of which shared memory returns 128 a clock,
// feed 96 or 128 multiply-adds, so that full the kernel does 32 TFLOP/s of 74 (8
// sequences of 1024 tokens, 32 heads of 128: 2.17 ms); 8 by 8 would leave one
// CTA of four warps on an SM.  Small calls are bound by a tile's latency
// instead: alone on an SM, with a warp per scheduler that issues an instruction in
// 2.8 clocks, it takes 6.7 us for 64 keys (D = 64; 12.0 at 128), so that keys are
// split over many CTAs.  Keys and values are
// copied in asynchronously: the next tile's keys beside this one's weights, its
// values beside the next scores.

#include <type_traits>

#include "extend_common.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFmaThreads = 128;

template <int D, int R>
struct FmaShape {
    static constexpr int RPT = R == 16 ? 4 : 8;             // rows of a thread
    static constexpr int TX = kFmaThreads * RPT / R;        // lanes that share them: 32 or 16
    static constexpr int KEYS = D == 128 && R == 64 ? 48 : 64;  // keys of a staged tile
    static constexpr int KPT = KEYS / TX;                   // keys of a thread
    static constexpr int CPT = D / TX;                      // columns of a thread
    static constexpr int smem = (R * (D + 4) + 2 * KEYS * (D + 4) + KEYS * (R + 4)) * 4 + KEYS * 4 + R * 16;
};

__device__ __forceinline__ void copy16(float *dst, const float *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all of this thread's copies but those of the newest group have arrived
__device__ __forceinline__ void copies_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Start to stage KEYS keys from k on of one pool into kv, as one group.  Rows
// from k1 on or in a block outside the pool are zero and, where bad is given,
// marked in it.
template <int D, int KEYS>
__device__ __forceinline__ void fma_stage(const ExtArgs &a, const float *pool, int seq, int kvh, int k,
                                          int k1, float *kv, int *bad) {
    constexpr int C = D / 4;
    const int shift = a.run_shift + 4;
#pragma unroll 2
    for (int i = threadIdx.x; i < KEYS * C; i += kFmaThreads) {
        const int r = i / C, c = i % C, j = k + r;
        float *dst = kv + r * (D + 4) + c * 4;
        bool ok = j < k1;
        if (ok) {
            const int b = __ldg(a.block_tables + (size_t)seq * a.max_blocks_per_seq + (j >> shift));
            ok = b >= 0 && b < a.num_blocks;
            if (ok)
                copy16(dst, pool + ((((size_t)b * a.num_kv_heads + kvh) << shift) + (j & ((1 << shift) - 1))) * D + c * 4);
            else if (c == 0 && bad)
                raise_fault(a.dev_error, PKV_FAULT_BLOCK_ID);
        }
        if (!ok) *reinterpret_cast<float4 *>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c == 0 && bad) bad[r] = !ok;
    }
    copies_commit();
}

// Whether a value that this thread staged is not finite.
template <int D, int KEYS>
__device__ __forceinline__ bool fma_odd(const float *kv) {
    constexpr int C = D / 4;
    bool odd = false;
#pragma unroll 4
    for (int i = threadIdx.x; i < KEYS * C; i += kFmaThreads) {
        const float4 v = *reinterpret_cast<const float4 *>(kv + (i / C) * (D + 4) + (i % C) * 4);
        odd |= !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w));
    }
    return odd;
}

// The score limited to (-cap, cap), in log2 units.
__device__ __noinline__ float fma_cap(float x, float cap) { return cap * tanhf(x / cap) * kLog2e; }

// Whether a node with this mask sees the tree's key `at` (negative: the context
// before the tree, which every node sees).
__device__ __noinline__ bool fma_tree_sees(const uint32_t *mask, int at, int nodes) {
    return at < 0 || (at < nodes && ((__ldg(mask + (at >> 5)) >> (at & 31)) & 1u));
}

// CTA: one tile of R rows, one kv head, one part of its keys.  A thread owns
// RPT rows; the TX lanes that share them split the keys of a score tile and
// the columns of the output.
template <int D, int R>
__global__ void __launch_bounds__(kFmaThreads) extend_fma_kernel(const ExtArgs a) {
    using S = FmaShape<D, R>;
    constexpr int RPT = S::RPT, TX = S::TX, KEYS = S::KEYS, KPT = S::KPT, CPT = S::CPT;
    constexpr int VEC = CPT < 4 ? CPT : 4;
    extern __shared__ __align__(16) float sm[];
    float *qs = sm, *ks = qs + R * (D + 4), *vs = ks + KEYS * (D + 4), *ps = vs + KEYS * (D + 4);
    int4 *sees = reinterpret_cast<int4 *>(ps + KEYS * (R + 4));  // a row's lo, hi, position, slope
    int *bad = reinterpret_cast<int *>(sees + R);
    const float *k_pool = static_cast<const float *>(a.k_pool), *v_pool = static_cast<const float *>(a.v_pool);
    griddep_launch();
    griddep_wait();
    ext_check_starts(a);
    const int kvh = blockIdx.x % a.num_kv_heads;
    __shared__ ExtTile tile;
    __shared__ int found;
    if (threadIdx.x < 32) {
        ExtTile t;
        int part;
        const bool ok = ext_find_item(a, blockIdx.x / a.num_kv_heads, R, t, part);
        if (threadIdx.x == 0) tile = t, found = ok ? part : -1;
    }
    __syncthreads();
    const ExtTile t = tile;
    const int part = found;
    if (part < 0) return;
    int k0, k1;
    ext_part(a, t, part, k0, k1);
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    const int G = a.group;
    fma_stage<D, KEYS>(a, k_pool, t.seq, kvh, k0, k1, ks, bad);
    fma_stage<D, KEYS>(a, v_pool, t.seq, kvh, k0, k1, vs, nullptr);
#pragma unroll 4
    for (int i = tid; i < R * (D / 4); i += kFmaThreads) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < t.nrows) {
            const int row = t.row0 + r, tok = row / G, g = row - tok * G;
            v = *reinterpret_cast<const float4 *>(
                static_cast<const float *>(a.q) +
                ((size_t)(t.q0 + tok) * a.num_heads + kvh * G + g) * D + c * 4);
        }
        *reinterpret_cast<float4 *>(qs + r * (D + 4) + c * 4) = v;
    }
    const int base = t.ctx - t.ntok;  // tree: key of node 0
    const int nodes = min(t.ntok, a.mask_words * 32);
    if (tid < R) {
        const int row = t.row0 + min(tid, t.nrows - 1), tok = row / G;
        int lo = 0, hi = base;  // a tree's nodes all see what was there before them
        if (!a.tree_mask) ext_row_range(a, t.prefix, base + tok, lo, hi);
        const float slope = a.slopes ? __ldg(a.slopes + kvh * G + row - tok * G) * kLog2e : 0.f;
        sees[tid] = make_int4(lo, hi, base + tok, __float_as_int(slope));
    }
    // keys that all rows of the tile see
    int seen_lo = 0, seen_hi = max(t.prefix, base + t.row0 / G + 1);
    if (a.window > 0) seen_lo = max(0, base + (t.row0 + t.nrows - 1) / G - a.window + 1);
    float m[RPT], l[RPT], o[RPT][CPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i] = -CUDART_INF_F, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CPT; ++c) o[i][c] = 0.f;
    }
    // (rows past the tile's last are computed like copies of it and not stored;
    // warps that have no others compute nothing)
    const bool busy = (tid & ~31) / TX * RPT < t.nrows;
    for (int k = k0; k < k1; k += KEYS) {
        copies_wait_but_one();
        __syncthreads();  // keys (and, first, queries) are there
        float s[RPT][KPT];
        if (busy) {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < KPT; ++j) s[i][j] = 0.f;
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                float4 kk[KPT];
#pragma unroll
                for (int j = 0; j < KPT; ++j)
                    kk[j] = *reinterpret_cast<const float4 *>(ks + (tx + j * TX) * (D + 4) + d);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float4 qv = *reinterpret_cast<const float4 *>(qs + (ty * RPT + i) * (D + 4) + d);
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        s[i][j] = fmaf(qv.x, kk[j].x, s[i][j]);
                        s[i][j] = fmaf(qv.y, kk[j].y, s[i][j]);
                        s[i][j] = fmaf(qv.z, kk[j].z, s[i][j]);
                        s[i][j] = fmaf(qv.w, kk[j].w, s[i][j]);
                    }
                }
            }
        }
        bool dead[KPT];
#pragma unroll
        for (int j = 0; j < KPT; ++j) dead[j] = bad[tx + j * TX];
        __syncthreads();  // keys are consumed
        fma_stage<D, KEYS>(a, k_pool, t.seq, kvh, k + KEYS, k1, ks, bad);
        if (busy) {
            // Each step is jumped over where the tile does not need it: code that
            // is laid out once per score is large, and fetching it costs more
            // than running it (512 keys for 512 rows, D = 128: 161 us with every
            // step in one loop, 129 so).
            const float unit = a.softcap > 0.f ? a.scale : a.scale * kLog2e;
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < KPT; ++j) s[i][j] *= unit;
            if (a.softcap > 0.f) {
#pragma unroll
                for (int i = 0; i < RPT; ++i)
#pragma unroll
                    for (int j = 0; j < KPT; ++j) s[i][j] = fma_cap(s[i][j], a.softcap);
            }
            if (a.slopes) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int4 see = sees[ty * RPT + i];
#pragma unroll
                    for (int j = 0; j < KPT; ++j)
                        s[i][j] -= __int_as_float(see.w) * fabsf((float)(see.z - (k + tx + j * TX)));
                }
            }
            if (a.tree_mask && k + KEYS > base) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const uint32_t *mask =
                        a.tree_mask + (size_t)(t.q0 + sees[ty * RPT + i].z - base) * a.mask_words;
#pragma unroll
                    for (int j = 0; j < KPT; ++j)
                        if (!fma_tree_sees(mask, k + tx + j * TX - base, nodes)) s[i][j] = -CUDART_INF_F;
                }
            } else if (!a.tree_mask && (k < seen_lo || k + KEYS > seen_hi)) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int4 see = sees[ty * RPT + i];
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        const int key = k + tx + j * TX;
                        if (key < see.x || key >= see.y) s[i][j] = -CUDART_INF_F;
                    }
                }
            }
            bool any_dead = false;
#pragma unroll
            for (int j = 0; j < KPT; ++j) any_dead |= dead[j];
            if (any_dead) {
#pragma unroll
                for (int j = 0; j < KPT; ++j)
#pragma unroll
                    for (int i = 0; i < RPT; ++i)
                        if (dead[j]) s[i][j] = -CUDART_INF_F;
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                float top = m[i];
                // a NaN score (its key is visible) is kept out of the maximum
                // and reaches the sums below
#pragma unroll
                for (int j = 0; j < KPT; ++j) top = fmaxf(top, s[i][j]);
#pragma unroll
                for (int x = TX / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float ref = top == -CUDART_INF_F ? 0.f : top;
                const float f = fast_exp2(m[i] - ref);  // 0 while m is -inf
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < KPT; ++j) {
                    s[i][j] = fast_exp2(s[i][j] - ref);
                    sum += s[i][j];
                }
                // (the lanes' sums are joined at the end)
                l[i] = l[i] * f + sum;
#pragma unroll
                for (int c = 0; c < CPT; ++c) o[i][c] *= f;
            }
#pragma unroll
            for (int j = 0; j < KPT; ++j)
#pragma unroll
                for (int i = 0; i < RPT; i += 4)
                    *reinterpret_cast<float4 *>(ps + (tx + j * TX) * (R + 4) + ty * RPT + i) =
                        make_float4(s[i][j], s[i + 1][j], s[i + 2][j], s[i + 3][j]);
        }
        copies_wait_but_one();
        // a value that is not finite must reach only the rows that see its key:
        // 0 * inf is NaN, so such a tile skips the weights that are zero
        const bool odd = __syncthreads_or(fma_odd<D, KEYS>(vs));  // weights and values are there
        auto add_values = [&](auto skip) {
#pragma unroll 2
            for (int j = 0; j < KEYS; ++j) {
                float p[RPT];
#pragma unroll
                for (int i = 0; i < RPT; i += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(ps + j * (R + 4) + ty * RPT + i);
                    p[i] = w.x, p[i + 1] = w.y, p[i + 2] = w.z, p[i + 3] = w.w;
                }
#pragma unroll
                for (int c = 0; c < CPT; c += VEC) {
                    const float *src = vs + j * (D + 4) + (c / VEC) * TX * VEC + tx * VEC;
                    float v[VEC];
                    if constexpr (VEC == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(src);
                        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2 *>(src);
                        v[0] = x.x, v[1] = x.y;
                    }
#pragma unroll
                    for (int i = 0; i < RPT; ++i)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (!decltype(skip)::value || p[i] != 0.f) o[i][c + e] = fmaf(p[i], v[e], o[i][c + e]);
                }
            }
        };
        if (busy && !odd) add_values(std::false_type());
        if (busy && odd) add_values(std::true_type());
        __syncthreads();  // values and weights are consumed
        fma_stage<D, KEYS>(a, v_pool, t.seq, kvh, k + KEYS, k1, vs, nullptr);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
        for (int x = TX / 2; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        const int r = ty * RPT + i;
        if (r >= t.nrows) continue;
        const int row = t.row0 + r, tok = row / G;
        const size_t oh = (size_t)(t.q0 + tok) * a.num_heads + kvh * G + row - tok * G;
        // l is NaN where a visible score was: the row is NaN, not empty
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const bool split = a.num_parts > 1;
        if (split && tx == 0)
            a.ws_lse[oh * a.num_parts + part] =
                l[i] == 0.f ? -CUDART_INF_F : m[i] + log2f(l[i]);
        if (split && l[i] == 0.f) continue;  // an empty part's output is not read
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int col = (c / VEC) * TX * VEC + tx * VEC + c % VEC;
            const float x = o[i][c] * inv;
            if (split)
                a.ws_o[(oh * a.num_parts + part) * D + col] = x;
            else
                store_out(a.out, oh * D + col, x, a.out_dtype);
        }
    }
}

template <int D, int R>
pkv_status launch_fma_one(const ExtLaunch &L) {
    auto kern = extend_fma_kernel<D, R>;
    constexpr int smem = FmaShape<D, R>::smem;
    static_assert(smem <= 227 * 1024, "shared memory budget");
    static unsigned long long done_mask = 0ull;
    const unsigned long long bit = 1ull << (L.device & 63);
    if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & bit)) {
        if (cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem)) != PKV_OK)
            return PKV_ERR_CUDA;
        __atomic_fetch_or(&done_mask, bit, __ATOMIC_RELEASE);
    }
    const dim3 grid((unsigned)L.args.tiles * L.args.num_kv_heads * L.args.num_parts);
    return cuda_status(launch_dependent(kern, grid, dim3(kFmaThreads), smem, L.stream, L.args));
}

template <int D>
pkv_status launch_fma_rows(const ExtLaunch &L) {
    return L.rows == 16 ? launch_fma_one<D, 16>(L) : launch_fma_one<D, 64>(L);
}

}  // namespace

pkv_status launch_extend_fma_f32(const ExtLaunch &L) {
    return L.head_dim == 64 ? launch_fma_rows<64>(L) : launch_fma_rows<128>(L);
}

}  // namespace pkv
