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
// Both directions are one launch, read each logit once and are bound by memory at large T * E.  W lanes
// (the least power of two with 16 values a lane, 32 for more than 512 experts) hold one token's row in
// registers, so the softmax takes one pass and a warp works on 32 / W tokens at once: with a warp to a token
// the shuffles of its sums were most of the instructions (16,384 x 128: 9.4 and 8.3 us, against 3.7 of
// memory time).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kBalSms = 152;
constexpr int kBalMaxChunks = 2 * kBalSms;   // forward: most blocks
constexpr int kBwdWarps = 8;
// forward: warps per block; two blocks an SM hold 32 warps where a warp has one row of up to 512 values at
// a time, which the memory needs then (131,072 x 512: 76 us with eight)
template <int W, int V>
constexpr int bal_warps() { return W == 32 && V == 16 ? 16 : 8; }
// blocks an SM: at most 64 registers for 16 values a lane, 128 for 32 (the backward of 131,072 x 512: 145 us
// with the 80 registers that the compiler would take, 102 with 64)
template <int V>
constexpr int bal_blocks_sm() { return V == 16 ? 4 : 2; }

__device__ __forceinline__ float bal_warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int W>
__device__ __forceinline__ float bal_group_sum(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Column of lane gl's value i (of W lanes): with 16-byte rows (E % 4 == 0) four consecutive columns per
// load, otherwise every W-th.
template <int W, bool VEC>
__device__ __forceinline__ int bal_col(int gl, int i) {
    return VEC ? 4 * (gl + W * (i >> 2)) + (i & 3) : gl + W * i;
}
// the lane's V values of a row; columns past E, and all of a row that is not there, read as -inf (p = 0)
template <int W, int V, bool VEC>
__device__ __forceinline__ void bal_load(float* x, const float* row, int E, int gl, bool there) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (there && bal_col<W, VEC>(gl, i) < E) v = __ldg(reinterpret_cast<const float4*>(row + bal_col<W, VEC>(gl, i)));
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = there && bal_col<W, VEC>(gl, i) < E ? __ldg(row + bal_col<W, VEC>(gl, i)) : -INFINITY;
    }
}
// Segment bounds, held inside [0, T]; without offsets one segment holds every token.
__device__ __forceinline__ int bal_off(const int* off, int s, int T) {
    return off ? min(max(__ldg(off + s), 0), T) : (s == 0 ? 0 : T);
}
// The first segment that ends after token t (B if none does), by the whole warp: up to 128 ends are looked at
// at once, since a search among them is a chain of loads.
__device__ __forceinline__ int bal_segment(const int* off, int B, int T, int t) {
    if (!off) return 0;   // one segment of all tokens
    if (B <= 128) {
        const int lane = threadIdx.x & 31;
        int s = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s += __popc(__ballot_sync(0xffffffffu, 32 * i + lane < B && bal_off(off, 32 * i + lane + 1, T) <= t));
        return s;
    }
    int lo = 0, hi = B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (bal_off(off, mid + 1, T) > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// e^x as a power of two, results below the least normal flushed to 0, which a softmax can do without
// (131,072 x 512: the forward 52.9 us with __expf, 50.1 so)
__device__ __forceinline__ float bal_exp(float x) { return exp2_approx(x * 1.442695041f); }

// The softmax of a group's row: x becomes exp(x - max).  A row of -inf alone has none: p = 0, lse taken as
// 0.  All lanes of the warp take part.
struct BalRow {
    float inv, lse;   // 1 / sum, log-sum-exp
    float max;
};
template <int W, int V>
__device__ __forceinline__ BalRow bal_softmax(float* x) {
    BalRow r;
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int o = W / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bool none = m == -INFINITY;
    if (__any_sync(0xffffffffu, none)) {   // fmaxf passes over NaN: a row of -inf and NaN is NaN
        int bad = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) bad |= isnan(x[i]);
#pragma unroll
        for (int o = W / 2; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
        none = none && !bad;
    }
    r.max = m;
    const float base = none ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = bal_exp(x[i] - base);   // 0 for -inf
        sum += x[i];
    }
    sum = bal_group_sum<W>(sum);
    r.inv = none ? 0.f : 1.f / sum;
    r.lse = none ? 0.f : m + logf(sum);
    return r;
}

// Forward.  Block c takes tokens [c chunk, (c+1) chunk), and of each segment that it meets sums p, the
// picks, lse^2 and the tokens: a piece.  A segment inside one block is finished there.  The pieces of a
// longer one are joined in `workspace`, where the sums of p are held as 64-bit integers, times the power of two
// that leaves their sum, at most T, below 2^62 (one that did for every T, 2^32, took the digits of picks with p
// under 1e-9), and the counts as integers: integers add up to the same in any order, and the block
// that comes last finishes the segment and leaves zeros for the next call.  The sums of lse^2, which have
// no such bound, are kept apart, one for each piece (block c's piece of segment s at c + s, which no other
// has: going through the tokens each block's end and each segment's end advances it by one), and added in
// order.  One launch: a second one that added 304 blocks' partial sums took 11 us at 128 experts.
//
// A block takes the segments that it meets one after the other, with four barriers and a sum over its warps each, so
// many short ones cost more than their tokens (131,072 x 128: 18 us with 1 segment, 27 with 1024, 69 with 8192, 590
// with 65,535; the backward 29, 31, 35, 46), and both directions pass empty segments one by one (65,533 of them in
// one place: 8 and 10 ms).
struct BalArgs {
    const float* logits;
    const int* idx;
    const uint8_t* mask;
    const int* off;
    int T, E, k, B, chunk;
    float fix, unfix;        // P's one, a power of two, and its inverse
    unsigned long long* P;   // [B, E] sum of p; all five are zero between calls, so that calls of other sizes may share
                             // the workspace
    int* C;                  // [B, E] picks
    int* N;                  // [B] counted tokens
    int* ticket;             // [B] pieces joined
    float* Z;                // [chunks + B] a piece's sum of lse^2
    int* counts;
    int* tokens;
    float* loss;
};

// Two sums over a block, whole on thread 0.
template <int kWarps>
__device__ __forceinline__ float2 bal_block_sum2(float a, float b, float2* part) {
    a = bal_warp_sum(a);
    b = bal_warp_sum(b);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 sum = make_float2(0.f, 0.f);
    if (threadIdx.x == 0)
        for (int w = 0; w < kWarps; ++w) {
            sum.x += part[w].x;
            sum.y += part[w].y;
        }
    return sum;
}

template <int W, int V, bool VEC>
__global__ void __launch_bounds__(32 * bal_warps<W, V>(), bal_blocks_sm<V>() * 8 / bal_warps<W, V>()) balance_fwd_kernel(const BalArgs a) {
    grid_dep_wait();
    constexpr int kWarps = bal_warps<W, V>();
    extern __shared__ float sm[];
    float* red = sm;                                            // [kWarps][E]
    int* hist = reinterpret_cast<int*>(red + kWarps * a.E);  // [E]
    __shared__ float part[kWarps];
    __shared__ float2 part2[kWarps];
    __shared__ int npart[kWarps];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane % W;
    const int t0 = blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    for (int s = bal_segment(a.off, a.B, a.T, t0); s < a.B; ++s) {
        const int s0 = bal_off(a.off, s, a.T), s1 = bal_off(a.off, s + 1, a.T);
        if (s0 >= t1) break;
        const int lo = max(s0, t0), hi = min(s1, t1);
        if (lo >= hi) continue;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
        // the thread's first two picks are under way while the tokens' rows are summed
        const long long p0 = (long long)lo * a.k + threadIdx.x, pe = (long long)hi * a.k;
        auto pick = [&](long long i) {
            const int e = i < pe ? __ldg(a.idx + i) : -1;
            return (unsigned)e < (unsigned)a.E && (!a.mask || __ldg(a.mask + (unsigned)i / (unsigned)a.k)) ? e : -1;
        };
        const int pick0 = pick(p0), pick1 = pick(p0 + 32 * kWarps);
        float acc[V], z2 = 0.f;
        int n = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        constexpr int G = 32 / W;   // tokens of a warp
        for (int tw = lo + warp * G; tw < hi; tw += kWarps * G) {
            const int t = tw + lane / W;
            const bool counts = t < hi && !(a.mask && !__ldg(a.mask + t));
            float x[V];
            bal_load<W, V, VEC>(x, a.logits + (long long)t * a.E, a.E, gl, counts);
            const BalRow r = bal_softmax<W, V>(x);   // (nothing where the token does not count)
            n += counts && gl == 0;
            z2 += gl == 0 ? r.lse * r.lse : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += x[i] * r.inv;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {   // the warp's tokens together; the first group holds them
#pragma unroll
            for (int o = W; o < 32; o *= 2) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            if (lane < W && bal_col<W, VEC>(gl, i) < a.E) red[warp * a.E + bal_col<W, VEC>(gl, i)] = acc[i];
        }
        z2 = bal_warp_sum(z2);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) {
            part[warp] = z2;
            npart[warp] = n;
        }
        __syncthreads();
        if (pick0 >= 0) atomicAdd(hist + pick0, 1);
        if (pick1 >= 0) atomicAdd(hist + pick1, 1);
        for (long long i = p0 + 64 * kWarps; i < pe; i += 32 * kWarps) {
            const int e = pick(i);
            if (e >= 0) atomicAdd(hist + e, 1);
        }
        z2 = 0.f;
        n = 0;
        for (int w = 0; w < kWarps; ++w) {
            z2 += part[w];
            n += npart[w];
        }
        __syncthreads();
        const bool whole = lo == s0 && hi == s1;
        unsigned long long* P = a.P + (long long)s * a.E;
        int* K = a.C + (long long)s * a.E;
        float dot = 0.f;   // sum_e c[e] sum_t p[t,e]
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[w * a.E + e];
            if (whole) {
                a.counts[(long long)s * a.E + e] = hist[e];
                dot += v * (float)hist[e];
            } else {
                atomicAdd(P + e, (unsigned long long)__float2ll_rn(v * a.fix));
                if (hist[e]) atomicAdd(K + e, hist[e]);
            }
        }
        bool finish = whole;
        if (!whole) {
            const int c0 = s0 / a.chunk, c1 = (s1 - 1) / a.chunk;   // the blocks that share the segment
            if (threadIdx.x == 0) {
                a.Z[blockIdx.x + s] = z2;
                atomicAdd(a.N + s, n);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                __threadfence();   // the block's sums, which the barrier orders before it, before its ticket
                last = atomicAdd(a.ticket + s, 1) == c1 - c0;
            }
            __syncthreads();
            finish = last;
            if (finish) {
                __threadfence();
                // requests first, so that their latencies overlap
                if (threadIdx.x == 0) {
                    n = atomicExch(a.N + s, 0);
                    a.ticket[s] = 0;
                }
                z2 = 0.f;
                for (int q = c0 + (int)threadIdx.x; q <= c1; q += blockDim.x) {
                    z2 += __ldcg(a.Z + q + s);
                    a.Z[q + s] = 0.f;
                }
                for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
                    const int c = atomicExch(K + e, 0);
                    const float v = __ll2float_rn((long long)atomicExch(P + e, 0ull)) * a.unfix;
                    a.counts[(long long)s * a.E + e] = c;
                    dot += v * (float)c;
                }
            }
        } else if (threadIdx.x != 0) {
            z2 = 0.f;   // every thread has the block's sum
        }
        if (finish) {
            const float2 sums = bal_block_sum2<kWarps>(dot, z2, part2);
            if (threadIdx.x == 0) {
                dot = sums.x;
                z2 = sums.y;
                const float inv = n > 0 ? 1.f / (float)n : 0.f;
                if (isnan(z2)) dot = z2;   // a NaN in a counted row: the integer sums do not show it
                a.tokens[s] = n;
                a.loss[2 * s] = (float)a.E / (float)a.k * inv * inv * dot;
                a.loss[2 * s + 1] = inv * z2;
            }
        }
        __syncthreads();   // the next segment's sums reuse the arrays
    }
    // a segment without tokens meets no block: the blocks share these out
    for (int s = blockIdx.x; s < a.B; s += gridDim.x)
        if (bal_off(a.off, s, a.T) >= bal_off(a.off, s + 1, a.T)) {
            for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[(long long)s * a.E + e] = 0;
            if (threadIdx.x == 0) {
                a.tokens[s] = 0;
                a.loss[2 * s] = a.loss[2 * s + 1] = 0.f;
            }
        }
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
    int T, E, k, B, rounds;
    float* dlogits;
};

// Each group of W lanes takes `rounds` tokens, a warp's groups neighbouring ones.
template <int W, int V, bool VEC>
__global__ void __launch_bounds__(32 * kBwdWarps, bal_blocks_sm<V>()) balance_bwd_kernel(const BalBwdArgs a) {
    grid_dep_wait();
    constexpr int G = 32 / W;
    const int lane = threadIdx.x & 31, gl = lane % W;
    const long long first = ((long long)blockIdx.x * kBwdWarps + (threadIdx.x >> 5)) * a.rounds * G;
    if (first >= a.T) return;
    int s = bal_segment(a.off, a.B, a.T, (int)first);
    int held = -1;
    float cf[V], scale = 0.f, zc = 0.f;   // db E / (k n^2) c[e] of the lane's columns, that factor, 2 dz / n
#pragma unroll
    for (int i = 0; i < V; ++i) cf[i] = 0.f;
    for (int q = 0; q < a.rounds; ++q) {
        const long long tw = first + (long long)q * G;
        if (tw >= a.T) break;
        const int t = (int)tw + lane / W;
        const bool live = t < a.T;
        const float* row = a.logits + (long long)t * a.E;
        float* out = a.dlogits + (long long)t * a.E;
        if (live)
            while (s < a.B && bal_off(a.off, s + 1, a.T) <= t) ++s;
        const bool counts = live && s < a.B && bal_off(a.off, s, a.T) <= t && !(a.mask && !__ldg(a.mask + t));
        float x[V];
        bal_load<W, V, VEC>(x, row, a.E, gl, counts);
        if (counts && held != s) {
            held = s;
            const int n = __ldg(a.tokens + s);
            const float inv = n > 0 ? 1.f / (float)n : 0.f;
            scale = __ldg(a.dloss + 2 * s) * ((float)a.E / (float)a.k) * inv * inv;
            zc = __ldg(a.dloss + 2 * s + 1) * 2.f * inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = bal_col<W, VEC>(gl, i);
                cf[i] = e < a.E ? scale * (float)__ldg(a.counts + (long long)s * a.E + e) : 0.f;
            }
        }
        const long long pk = (long long)t * a.k;
        float wdw = 0.f;
        if (a.w && live)
            for (int j = gl; j < a.k; j += W) wdw += __ldg(a.w + pk + j) * __ldg(a.dw + pk + j);
        wdw = bal_group_sum<W>(wdw);
        __syncwarp();
        const BalRow r = bal_softmax<W, V>(x);   // x is 0 where the token does not count
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) dot += x[i] * cf[i];
        dot = bal_group_sum<W>(dot);
        const float shift = (zc * r.lse - dot * r.inv) * r.inv;
        if (live) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = counts ? x[i] * (r.inv * cf[i] + shift) : 0.f;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    if (bal_col<W, VEC>(gl, i) < a.E)
                        *reinterpret_cast<float4*>(out + bal_col<W, VEC>(gl, i)) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (bal_col<W, VEC>(gl, i) < a.E) out[bal_col<W, VEC>(gl, i)] = x[i];
            }
        }
        __syncwarp();   // the row's values are ordered before the picks' that replace them
        if (a.w && live)
            for (int j = gl; j < a.k; j += W) {
                const int e = __ldg(a.idx + pk + j);
                if ((unsigned)e >= (unsigned)a.E) continue;
                float v = __ldg(a.w + pk + j) * (__ldg(a.dw + pk + j) - wdw);
                if (counts && r.inv != 0.f)
                    v += bal_exp(__ldg(row + e) - r.max) *
                         (r.inv * scale * (float)__ldg(a.counts + (long long)s * a.E + e) + shift);
                out[e] = v;
            }
    }
}

// ---- launches --------------------------------------------------------------------------------------
// Tokens of a block: two rounds of its warps at least (a join of two blocks costs more: 64 x 128 took 5.5 us
// in two blocks)
static int bal_chunk(int64_t T, int64_t E) {
    const int64_t least = E <= 16 ? 512 : E <= 32 ? 256 : E <= 64 ? 128 : 64;
    return (int)std::max<int64_t>(least, (T + kBalMaxChunks - 1) / kBalMaxChunks);
}
static size_t bal_blocks(int64_t T, int64_t E) { return (size_t)((T + bal_chunk(T, E) - 1) / bal_chunk(T, E)); }

// the status word's line, then P, C, N, ticket, Z
size_t balance_workspace(int64_t T, int64_t E, int64_t B) {
    return 256 + (size_t)B * (12 * (size_t)E + 8) + 4 * (bal_blocks(T, E) + (size_t)B);
}

template <int W, int V, bool VEC>
static cudaError_t fwd_c(cudaStream_t st, const BalArgs& a) {
    constexpr int kWarps = bal_warps<W, V>();
    const size_t smem = (size_t)(kWarps + 1) * a.E * 4;   // at most 36 KB
    // (with no tokens one block writes the zeros)
    return launch_pdl(balance_fwd_kernel<W, V, VEC>, (unsigned)std::max<size_t>(1, bal_blocks(a.T, a.E)), 32 * kWarps, smem, st, a);
}
template <int W, int V, bool VEC>
static cudaError_t bwd_c(cudaStream_t st, BalBwdArgs a) {
    // as many warps as the GPU holds at 32 an SM, each with so many rounds of tokens
    constexpr int G = 32 / W;
    const int groups = (a.T + G - 1) / G;
    a.rounds = std::max(1, (groups + kBalSms * 32 - 1) / (kBalSms * 32));
    const int warps = (groups + a.rounds - 1) / a.rounds;
    return launch_pdl(balance_bwd_kernel<W, V, VEC>, (warps + kBwdWarps - 1) / kBwdWarps, 32 * kBwdWarps, 0, st, a);
}
// lanes a token and values a lane
#define MOE_BAL_DISPATCH_VEC(fn, a, VEC)                    \
    if ((a).E <= 16) return fn<1, 16, VEC>(st, a);          \
    if ((a).E <= 32) return fn<2, 16, VEC>(st, a);          \
    if ((a).E <= 64) return fn<4, 16, VEC>(st, a);          \
    if ((a).E <= 128) return fn<8, 16, VEC>(st, a);         \
    if ((a).E <= 256) return fn<16, 16, VEC>(st, a);        \
    if ((a).E <= 512) return fn<32, 16, VEC>(st, a);        \
    return fn<32, 32, VEC>(st, a);
// four values at a time where rows are 16-byte aligned
#define MOE_BAL_DISPATCH(fn, a)                             \
    if ((a).E % 4 == 0) { MOE_BAL_DISPATCH_VEC(fn, a, true) } \
    MOE_BAL_DISPATCH_VEC(fn, a, false)

static cudaError_t dispatch_fwd(cudaStream_t st, const BalArgs& a) { MOE_BAL_DISPATCH(fwd_c, a) }
static cudaError_t dispatch_bwd(cudaStream_t st, const BalBwdArgs& a) { MOE_BAL_DISPATCH(bwd_c, a) }

cudaError_t launch_balance_fwd(cudaStream_t st, const float* logits, const int* topk_idx, const uint8_t* mask,
                               const int* seg_offsets, int T, int E, int k, int B, int* counts, int* tokens, float* loss,
                               void* workspace) {
    BalArgs a{logits, topk_idx, mask, seg_offsets, T, E, k, B, bal_chunk(T, E), (float)(1ull << 62)};
    for (int64_t most = 1; most < T; most *= 2) a.fix *= 0.5f;
    a.unfix = 1.f / a.fix;
    char* w = static_cast<char*>(workspace) + 256;
    const size_t be = (size_t)B * E;
    a.P = reinterpret_cast<unsigned long long*>(w);
    a.C = reinterpret_cast<int*>(w + be * 8);
    a.N = a.C + be;
    a.ticket = a.N + B;
    a.Z = reinterpret_cast<float*>(a.ticket + B);
    a.counts = counts;
    a.tokens = tokens;
    a.loss = loss;
    return dispatch_fwd(st, a);
}

cudaError_t launch_balance_bwd(cudaStream_t st, const float* logits, const int* topk_idx, const float* topk_w,
                               const float* dtopk_w, const uint8_t* mask, const int* seg_offsets, const int* counts,
                               const int* tokens, const float* dloss, int T, int E, int k, int B, float* dlogits) {
    if (T == 0) return cudaSuccess;
    const BalBwdArgs a{logits, topk_idx, topk_w, dtopk_w, mask, seg_offsets, counts, tokens, dloss, T, E, k, B, 0, dlogits};
    return dispatch_bwd(st, a);
}

}  // namespace moe
