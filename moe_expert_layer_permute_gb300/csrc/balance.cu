// balance.cu - the router's balance loss, z-loss and per-expert counts for each segment of a batch,
// and their gradient, joined with the gradient of the top-k weights.
//
// With l the logits [T, E], p[t] = softmax(l[t]), lse[t] its log-sum-exp, and over the counted tokens
// of segment s (mask set, seg_offsets[s] <= t < seg_offsets[s+1]) n their number and c[e] the picks of
// expert e among their k:
//   loss[s] = (E / (k n^2) sum_e c[e] sum_t p[t,e],  1/n sum_t lse[t]^2)          (0, 0 where n = 0)
//   dl[t,e] = db E / (k n^2) p[t,e] (c[e] - sum_i c[i] p[t,i]) + dz 2/n lse[t] p[t,e]
//             + w_j (dw_j - sum_i w_i dw_i) where e is the token's pick j
// The counts carry no gradient.
//
// Both directions read each logit once and are bound by memory at large T * E and by launches below.
// A warp holds one token's row in registers (E / 32 values a lane), so the softmax takes one pass.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kBalWarps = 16;         // forward: warps (tokens in flight) per block
constexpr int kBalMaxChunks = 304;    // forward: most blocks (two per SM)
constexpr int kBalMinChunk = 32;      // forward: fewest tokens per block
constexpr int kFinCols = 128;         // finish: columns per block
constexpr int kFinGroups = 8;         // finish: slot groups per block
constexpr int kBwdWarps = 8;

__device__ __forceinline__ float bal_warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float bal_warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Column of a lane's value i: with 16-byte rows (E % 4 == 0) four consecutive columns per load,
// otherwise every 32nd.
template <bool VEC>
__device__ __forceinline__ int bal_col(int lane, int i) {
    return VEC ? 4 * (lane + 32 * (i >> 2)) + (i & 3) : lane + 32 * i;
}
// the lane's C values of a row; columns past E read as -inf (p = 0)
template <int C, bool VEC>
__device__ __forceinline__ void bal_load(float* x, const float* row, int E, int lane) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (bal_col<VEC>(lane, i) < E) v = __ldg(reinterpret_cast<const float4*>(row + bal_col<VEC>(lane, i)));
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = bal_col<VEC>(lane, i) < E ? __ldg(row + bal_col<VEC>(lane, i)) : -INFINITY;
    }
}
// Segment bounds, held inside [0, T]; without offsets one segment holds every token.
__device__ __forceinline__ int bal_off(const int* off, int s, int T) {
    return off ? min(max(__ldg(off + s), 0), T) : (s == 0 ? 0 : T);
}
// the first segment that ends after token t (B if none does)
__device__ __forceinline__ int bal_segment(const int* off, int B, int T, int t) {
    int lo = 0, hi = B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (bal_off(off, mid + 1, T) > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// Block c takes tokens [c chunk, (c+1) chunk) and writes one slot of sums for each segment that it
// meets.  Going through the tokens in order, each chunk end and each segment end advances the slot
// by one, so slot c + s belongs to this pair alone and chunks + B slots hold them all: no atomics on
// floats, and sums in an order that depends on the sizes only.
struct BalArgs {
    const float* logits;
    const int* idx;
    const uint8_t* mask;
    const int* off;
    int T, E, k, B, chunk;
    float* P;      // [slots, E] sum of p
    int* C;        // [slots, E] picks
    float* Z;      // [slots] sum of lse^2
    int* N;        // [slots] counted tokens
};

template <int C, bool VEC>
__global__ void __launch_bounds__(32 * kBalWarps) balance_fwd_kernel(const BalArgs a) {
    grid_dep_wait();
    extern __shared__ float sm[];
    float* red = sm;                                            // [kBalWarps][E]
    int* hist = reinterpret_cast<int*>(red + kBalWarps * a.E);  // [E]
    __shared__ float zred[kBalWarps];
    __shared__ int nred[kBalWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    for (int s = bal_segment(a.off, a.B, a.T, t0); s < a.B; ++s) {
        const int s0 = bal_off(a.off, s, a.T);
        if (s0 >= t1) break;
        const int lo = max(s0, t0), hi = min(bal_off(a.off, s + 1, a.T), t1);
        if (lo >= hi) continue;
        const long long slot = blockIdx.x + s;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
        float acc[C];
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = 0.f;
        float z2 = 0.f;
        int n = 0;
        for (int t = lo + warp; t < hi; t += kBalWarps) {
            if (a.mask && !__ldg(a.mask + t)) continue;
            ++n;
            float x[C];
            bal_load<C, VEC>(x, a.logits + (long long)t * a.E, a.E, lane);
            float m = x[0];
#pragma unroll
            for (int i = 1; i < C; ++i) m = fmaxf(m, x[i]);
            m = bal_warp_max(m);
            float sum = 0.f;
            // a row of -inf alone has no softmax: p = 0, and nothing is added to either loss
            const bool none = m == -INFINITY;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                x[i] = none ? 0.f : __expf(x[i] - m);
                sum += x[i];
            }
            sum = bal_warp_sum(sum);
            const float inv = none ? 0.f : 1.f / sum;
            const float lse = none ? 0.f : m + logf(sum);
            z2 += lse * lse;
#pragma unroll
            for (int i = 0; i < C; ++i) acc[i] += x[i] * inv;
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (bal_col<VEC>(lane, i) < a.E) red[warp * a.E + bal_col<VEC>(lane, i)] = acc[i];
        if (lane == 0) {
            zred[warp] = z2;
            nred[warp] = n;
        }
        __syncthreads();
        for (long long i = (long long)lo * a.k + threadIdx.x; i < (long long)hi * a.k; i += blockDim.x) {
            const int e = __ldg(a.idx + i);
            if ((unsigned)e < (unsigned)a.E && (!a.mask || __ldg(a.mask + i / a.k))) atomicAdd(hist + e, 1);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) v += red[w * a.E + e];
            a.P[slot * a.E + e] = v;
            a.C[slot * a.E + e] = hist[e];
        }
        if (threadIdx.x == 0) {
            float v = 0.f;
            int c = 0;
            for (int w = 0; w < kBalWarps; ++w) {
                v += zred[w];
                c += nred[w];
            }
            a.Z[slot] = v;
            a.N[slot] = c;
        }
        __syncthreads();   // the next segment's sums reuse the arrays
    }
}

// Segment blockIdx.y: a cluster of ceil(E / 128) blocks, 128 columns each, adds the segment's slots
// (eight groups of threads take every eighth, then the groups in order) and the first block joins the
// blocks' parts of sum_e c[e] P[e] through distributed shared memory, in their order.
__global__ void __launch_bounds__(kFinCols * kFinGroups) balance_finish_kernel(const BalArgs a, int* counts, int* tokens,
                                                                              float* loss) {
    grid_dep_wait();
    __shared__ float sp[kFinGroups][kFinCols];
    __shared__ int sc[kFinGroups][kFinCols];
    __shared__ float sz[kFinCols * kFinGroups / 32];
    __shared__ int sn[kFinCols * kFinGroups / 32];
    __shared__ float part;
    const int s = blockIdx.y, rank = blockIdx.x, blocks = gridDim.x;
    const int col = threadIdx.x % kFinCols, grp = threadIdx.x / kFinCols;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = rank * kFinCols + col;
    const int lo = bal_off(a.off, s, a.T), hi = bal_off(a.off, s + 1, a.T);
    const int c0 = lo / a.chunk, c1 = hi > lo ? (hi - 1) / a.chunk : c0 - 1;
    float p = 0.f, z = 0.f;
    int c = 0, n = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int q = c0 + grp; q <= c1; q += kFinGroups) {
            const long long at = (long long)(q + s) * a.E + e;
            p += a.P[at];
            c += a.C[at];
        }
    }
    for (int q = c0 + (int)threadIdx.x; q <= c1; q += blockDim.x) {
        z += a.Z[q + s];
        n += a.N[q + s];
    }
    sp[grp][col] = p;
    sc[grp][col] = c;
    z = bal_warp_sum(z);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
        sz[warp] = z;
        sn[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        z = bal_warp_sum(sz[lane]);
        n = __reduce_add_sync(0xffffffffu, sn[lane]);
        float mine = 0.f;
        for (int j = lane; j < kFinCols; j += 32) {
            float v = 0.f;
            int k = 0;
#pragma unroll
            for (int g = 0; g < kFinGroups; ++g) {
                v += sp[g][j];
                k += sc[g][j];
            }
            if (rank * kFinCols + j < a.E) {
                counts[(long long)s * a.E + rank * kFinCols + j] = k;
                mine += v * (float)k;
            }
        }
        mine = bal_warp_sum(mine);
        if (lane == 0) part = mine;
    }
    if (blocks > 1) cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        float total = part;
        for (int b = 1; b < blocks; ++b) total += ld_cluster_f32(cluster_addr(&part, b));
        const float inv = n > 0 ? 1.f / (float)n : 0.f;
        tokens[s] = n;
        loss[2 * s] = (float)a.E / (float)a.k * inv * inv * total;
        loss[2 * s + 1] = inv * z;
    }
    if (blocks > 1) cluster_sync();   // the first block has read the others' parts before they exit
}

struct BalBwdArgs {
    const float* logits;
    const int* idx;
    const float* w;      // null together with dw: no top-k weights' gradient
    const float* dw;
    const uint8_t* mask;
    const int* off;
    const int* counts;
    const int* tokens;
    const float* dloss;
    int T, E, k, B, per_warp;
    float* dlogits;
};

// One warp takes per_warp consecutive tokens and keeps its columns' share of the segment's counts,
// db E / (k n^2) c[e], in registers while the segment lasts.
template <int C, bool VEC>
__global__ void __launch_bounds__(32 * kBwdWarps) balance_bwd_kernel(const BalBwdArgs a) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const long long first = ((long long)blockIdx.x * kBwdWarps + (threadIdx.x >> 5)) * a.per_warp;
    if (first >= a.T) return;
    const int t1 = (int)min((long long)a.T, first + a.per_warp);
    int s = bal_segment(a.off, a.B, a.T, (int)first);
    int held = -1;
    float cf[C], scale = 0.f, zc = 0.f;
    for (int t = (int)first; t < t1; ++t) {
        while (s < a.B && bal_off(a.off, s + 1, a.T) <= t) ++s;
        const bool counted = s < a.B && bal_off(a.off, s, a.T) <= t && !(a.mask && !__ldg(a.mask + t));
        float* out = a.dlogits + (long long)t * a.E;
        // the pick of this lane, and the top-k weights' gradient at it
        int pick = -1;
        float add = 0.f;
        if (a.w) {
            float w = 0.f, dw = 0.f;
            if (lane < a.k) {
                pick = __ldg(a.idx + (long long)t * a.k + lane);
                w = __ldg(a.w + (long long)t * a.k + lane);
                dw = __ldg(a.dw + (long long)t * a.k + lane);
            }
            add = w * (dw - bal_warp_sum(w * dw));
            if ((unsigned)pick >= (unsigned)a.E) pick = -1;
        }
        float x[C];
        if (counted) {
            const float* row = a.logits + (long long)t * a.E;
            if (held != s) {
                held = s;
                const int n = __ldg(a.tokens + s);
                const float inv = n > 0 ? 1.f / (float)n : 0.f;
                scale = __ldg(a.dloss + 2 * s) * ((float)a.E / (float)a.k) * inv * inv;
                zc = __ldg(a.dloss + 2 * s + 1) * 2.f * inv;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int e = bal_col<VEC>(lane, i);
                    cf[i] = e < a.E ? scale * (float)__ldg(a.counts + (long long)s * a.E + e) : 0.f;
                }
            }
            bal_load<C, VEC>(x, row, a.E, lane);
            const float at_pick = pick >= 0 ? __ldg(row + pick) : 0.f;
            float m = x[0];
#pragma unroll
            for (int i = 1; i < C; ++i) m = fmaxf(m, x[i]);
            m = bal_warp_max(m);
            const bool none = m == -INFINITY;
            float sum = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                x[i] = none ? 0.f : __expf(x[i] - m);
                sum += x[i];
                dot += x[i] * cf[i];
            }
            sum = bal_warp_sum(sum);
            dot = bal_warp_sum(dot);
            const float inv = none ? 0.f : 1.f / sum;
            const float shift = none ? 0.f : zc * (m + logf(sum)) - dot * inv;
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = x[i] * inv * (cf[i] + shift);
            if (pick >= 0 && !none)
                add += __expf(at_pick - m) * inv * (scale * (float)__ldg(a.counts + (long long)s * a.E + pick) + shift);
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = 0.f;
        }
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < C; i += 4)
                if (bal_col<VEC>(lane, i) < a.E)
                    *reinterpret_cast<float4*>(out + bal_col<VEC>(lane, i)) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (bal_col<VEC>(lane, i) < a.E) out[bal_col<VEC>(lane, i)] = x[i];
        }
        __syncwarp();   // the row's values are ordered before the picks' that replace them
        if (pick >= 0) out[pick] = add;
    }
}

// ---- launches --------------------------------------------------------------------------------------
static int bal_chunk(int64_t T) {
    return (int)std::max<int64_t>(kBalMinChunk, (T + kBalMaxChunks - 1) / kBalMaxChunks);
}
static int64_t bal_slots(int64_t T, int64_t B) { return (T + bal_chunk(T) - 1) / bal_chunk(T) + B; }

size_t balance_workspace(int64_t T, int64_t E, int64_t B) {
    return (size_t)256 + (size_t)bal_slots(T, B) * (8 * (size_t)E + 8);   // 256: the status word's line
}

template <int C, bool VEC>
static cudaError_t fwd_c(cudaStream_t st, const BalArgs& a) {
    const size_t smem = (size_t)(kBalWarps + 1) * a.E * 4;
    if constexpr (C == 32) {   // up to 68 KB; the smaller ones stay below 48 KB
        static const cudaError_t err =
            cudaFuncSetAttribute(balance_fwd_kernel<C, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (kBalWarps + 1) * 32 * C * 4);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(balance_fwd_kernel<C, VEC>, (a.T + a.chunk - 1) / a.chunk, 32 * kBalWarps, smem, st, a);
}
template <int C, bool VEC>
static cudaError_t bwd_c(cudaStream_t st, const BalBwdArgs& a) {
    const int warps = (a.T + a.per_warp - 1) / a.per_warp;
    return launch_pdl(balance_bwd_kernel<C, VEC>, (warps + kBwdWarps - 1) / kBwdWarps, 32 * kBwdWarps, 0, st, a);
}
// values per lane: four at a time where rows are 16-byte aligned
#define MOE_BAL_DISPATCH(fn, a)                         \
    if ((a).E % 4 == 0) {                               \
        if ((a).E <= 128) return fn<4, true>(st, a);    \
        if ((a).E <= 256) return fn<8, true>(st, a);    \
        if ((a).E <= 512) return fn<16, true>(st, a);   \
        return fn<32, true>(st, a);                     \
    }                                                   \
    if ((a).E <= 32) return fn<1, false>(st, a);        \
    if ((a).E <= 64) return fn<2, false>(st, a);        \
    if ((a).E <= 128) return fn<4, false>(st, a);       \
    if ((a).E <= 256) return fn<8, false>(st, a);       \
    if ((a).E <= 512) return fn<16, false>(st, a);      \
    return fn<32, false>(st, a);

static cudaError_t dispatch_fwd(cudaStream_t st, const BalArgs& a) { MOE_BAL_DISPATCH(fwd_c, a) }
static cudaError_t dispatch_bwd(cudaStream_t st, const BalBwdArgs& a) { MOE_BAL_DISPATCH(bwd_c, a) }

cudaError_t launch_balance_fwd(cudaStream_t st, const float* logits, const int* topk_idx, const uint8_t* mask,
                               const int* seg_offsets, int T, int E, int k, int B, int* counts, int* tokens, float* loss,
                               void* workspace) {
    BalArgs a{logits, topk_idx, mask, seg_offsets, T, E, k, B, bal_chunk(T)};
    const size_t slots = bal_slots(T, B);
    char* w = static_cast<char*>(workspace) + 256;
    a.P = reinterpret_cast<float*>(w);
    a.C = reinterpret_cast<int*>(w + slots * E * 4);
    a.Z = reinterpret_cast<float*>(w + slots * E * 8);
    a.N = reinterpret_cast<int*>(w + slots * E * 8 + slots * 4);
    if (T > 0) {
        const cudaError_t err = dispatch_fwd(st, a);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (E + kFinCols - 1) / kFinCols;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((E + kFinCols - 1) / kFinCols, B);
    cfg.blockDim = dim3(kFinCols * kFinGroups);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, balance_finish_kernel, a, counts, tokens, loss);
}

cudaError_t launch_balance_bwd(cudaStream_t st, const float* logits, const int* topk_idx, const float* topk_w,
                               const float* dtopk_w, const uint8_t* mask, const int* seg_offsets, const int* counts,
                               const int* tokens, const float* dloss, int T, int E, int k, int B, float* dlogits) {
    if (T == 0) return cudaSuccess;
    // as many warps as the GPU holds at 32 warps an SM (152 SMs), each with a run of tokens
    const int per_warp = std::max(1, (T + 152 * 32 - 1) / (152 * 32));
    const BalBwdArgs a{logits, topk_idx, topk_w, dtopk_w, mask, seg_offsets, counts, tokens, dloss, T, E, k, B, per_warp,
                       dlogits};
    return dispatch_bwd(st, a);
}

}  // namespace moe
