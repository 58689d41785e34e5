// select.cu - routing by scores: launches of the forward (select_fwd.cuh), the weights' gradient, and the step that moves the
// bias.
#include "select_fwd.cuh"
#include "per_device.h"

namespace moe {

extern template cudaError_t select_kind<kSelOdd>(cudaStream_t, const SelectArgs&, int, int, int);
extern template cudaError_t select_kind<kSelVec>(cudaStream_t, const SelectArgs&, int, int, int);
extern template cudaError_t select_kind<kSelFull>(cudaStream_t, const SelectArgs&, int, int, int);

// ---- backward --------------------------------------------------------------------------------------------------
// With D = sum_i w_i dw_i over the picks:
//   sigmoid                 dl_j = w_j (dw_j - D / scale) (1 - s_j), without the D where weights are not renormalised
//   softmax, renormalised   dl_j = w_j (dw_j - D / scale)
//   softmax, not            dl_e = -s_e D, and + w_j dw_j at the picks
// The first two touch the picks alone: a warp keeps two tiles of zeros in shared memory, puts a tile's picks in, sends it
// off as one bulk copy (tokens' rows follow one another) and takes the picks out again, so that a row costs k stores
// and no instruction for its zeros.  A tile's time is that of two loads, one after the other, and memory is kept busy by
// the tiles of twelve and more warps an SM (131,072 x 512, k = 8: a block to a tile, with its barriers, took 68 us).
struct SelItem {              // pick j of a token, over kp lanes of it
    int e;                    // -1: none
    float w, dw, x;
};
__device__ __forceinline__ SelItem sel_pick_of(const SelectGradArgs& a, long long t, int j, bool on) {
    SelItem g{-1, 0.f, 0.f, 0.f};
    if (on) {
        g.e = __ldg(a.idx + t * a.k + j);
        g.w = __ldg(a.w + t * a.k + j);
        g.dw = __ldg(a.dw + t * a.k + j);
    }
    return g;
}
__device__ __forceinline__ void sel_logit_of(const SelectGradArgs& a, long long t, SelItem& g) {
    if ((unsigned)g.e >= (unsigned)a.E) g.e = -1;
    if (g.e >= 0 && a.sigmoid)
        g.x = a.bf16 ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(a.logits) + t * a.E + g.e))
                     : __ldg(static_cast<const float*>(a.logits) + t * a.E + g.e);
}
__device__ __forceinline__ float sel_grad(const SelectGradArgs& a, SelItem g, int kp) {
    if (g.e < 0) g.w = g.dw = 0.f;   // (whatever stands beside no pick)
    float D = 0.f;
    if (a.renorm) {
        // less the heaviest pick's dw throughout, which the weights' sum of `scale` leaves as it was: a token of which one
        // pick has nearly all the weight keeps the digits of what is left
        const int first = (threadIdx.x & 31) & ~(kp - 1);
        const uint32_t heaviest = __ballot_sync(0xffffffffu, g.w == sel_segment_max(g.w, kp)) >> first;
        const float dw0 = __shfl_sync(0xffffffffu, g.dw, first + (heaviest ? __ffs(heaviest) - 1 : 0) % kp);
        if (g.e >= 0) g.dw -= dw0;
        D = sel_segment_sum(g.w * g.dw, kp) * a.inv_scale;
    }
    const float keep = a.sigmoid ? 1.f / (1.f + expf(g.x)) : 1.f;
    return g.w * (g.dw - D) * keep;
}

constexpr int kSparseWarps = 4;

template <bool BF>
__global__ void __launch_bounds__(32 * kSparseWarps) select_bwd_sparse_kernel(const SelectGradArgs a) {
    grid_dep_wait();
    using V = std::conditional_t<BF, __nv_bfloat16, float>;
    extern __shared__ __align__(128) unsigned char sel_tiles[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tile_bytes = (uint32_t)a.tile * a.E * sizeof(V);     // a multiple of 16
    V* const tiles = reinterpret_cast<V*>(sel_tiles + warp * 2 * tile_bytes);
    int* const spots = reinterpret_cast<int*>(sel_tiles + kSparseWarps * 2 * tile_bytes) + warp * 2 * a.tile * a.k;   // of the picks
    int kp = 1;
    while (kp < a.k) kp *= 2;
    const int per = 32 / kp, j = lane & (kp - 1), mine = lane / kp;
    const bool once = a.tile <= per;   // a lane has one pick of a tile: those of the next two are under way meanwhile
    // from the last tile to the first: the logits that a forward has read last may still be in L2
    const long long stride = -(long long)gridDim.x * kSparseWarps;
    long long tile = (a.T - 1) / a.tile - ((long long)blockIdx.x * kSparseWarps + warp);
    auto token = [&](long long of, int tk) { return of * a.tile + tk; };
    auto there = [&](long long of, int tk) { return of >= 0 && tk < a.tile && j < a.k && token(of, tk) < a.T; };
    SelItem now{}, next{};
    if (once) {
        now = sel_pick_of(a, token(tile, mine), j, there(tile, mine));
        next = sel_pick_of(a, token(tile + stride, mine), j, there(tile + stride, mine));
        sel_logit_of(a, token(tile, mine), now);
    }
    for (int n = 0; tile >= 0; tile += stride, ++n) {
        const long long t0 = tile * a.tile;
        const int tokens = (int)min((long long)a.tile, a.T - t0), slot = n & 1;
        V* const buf = tiles + slot * a.tile * a.E;
        int* const spot = spots + slot * a.tile * a.k;
        if (n < 2) {
            for (uint32_t i = lane * 16; i < tile_bytes; i += 32 * 16)
                *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(buf) + i) = make_uint4(0, 0, 0, 0);
        } else {   // the copy of two tiles ago has been read; its picks go
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
            for (int i = lane; i < a.tile * a.k; i += 32)
                if (spot[i] >= 0) buf[spot[i]] = V(0.f);
        }
        __syncwarp();
        auto place = [&](const SelItem& g, int tk) {
            const float d = sel_grad(a, g, kp);
            const int at = g.e >= 0 ? tk * a.E + g.e : -1;
            if (at >= 0) buf[at] = V(d);
            if (tk < a.tile && j < a.k) spot[tk * a.k + j] = at;
        };
        if (once) {
            sel_logit_of(a, token(tile + stride, mine), next);
            const SelItem after = sel_pick_of(a, token(tile + 2 * stride, mine), j, there(tile + 2 * stride, mine));
            place(now, mine);
            now = next;
            next = after;
        } else {
            for (int q = 0; q < a.tile; q += per) {
                const int tk = q + mine;
                SelItem g = sel_pick_of(a, token(tile, tk), j, there(tile, tk));
                sel_logit_of(a, token(tile, tk), g);
                place(g, tk);
            }
        }
        fence_proxy_async_cta();
        __syncwarp();
        unsigned char* out = static_cast<unsigned char*>(a.dlogits) + t0 * a.E * (long long)sizeof(V);
        const uint32_t bytes = (uint32_t)tokens * a.E * sizeof(V), whole = bytes & ~15u;
        if (lane == 0) {
            if (whole) bulk_store(out, buf, whole);
            bulk_commit();
        }
        if (lane * 2 < bytes - whole)   // the last tile's end
            reinterpret_cast<uint16_t*>(out + whole)[lane] = reinterpret_cast<const uint16_t*>(reinterpret_cast<unsigned char*>(buf) + whole)[lane];
    }
    if (lane == 0) bulk_wait_all();
}

// dlogits += the gradient where only picks have one
__global__ void __launch_bounds__(256) select_bwd_add_kernel(const SelectGradArgs a) {
    grid_dep_wait();
    int kp = 1;
    while (kp < a.k) kp *= 2;
    const int lane = threadIdx.x & 31, per = 32 / kp;
    const long long t = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * per + lane / kp;
    const int j = lane & (kp - 1);
    SelItem g = sel_pick_of(a, t, j, t < a.T && j < a.k);
    sel_logit_of(a, t, g);
    const float d = sel_grad(a, g, kp);
    if (g.e >= 0) static_cast<float*>(a.dlogits)[t * a.E + g.e] += d;
}

template <int W, int V, bool VEC>
__global__ void __launch_bounds__(256, V == 16 ? 4 : 2) select_bwd_dense_kernel(const SelectGradArgs a) {
    grid_dep_wait();
    constexpr int NT = 32 / W;
    const int lane = threadIdx.x & 31, gl = lane % W;
    SelectArgs row{};
    row.logits = a.logits;
    row.bf16 = a.bf16;
    const long long step = (long long)gridDim.x * 8 * NT;
    for (long long first = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * NT; first < a.T; first += step) {
        const long long t = first + lane / W;
        const bool live = t < a.T;
        float D = 0.f;
        bool any = false;
        for (int j = gl; live && j < a.k; j += W) {
            const int e = __ldg(a.idx + t * a.k + j);
            if ((unsigned)e < (unsigned)a.E) {
                D += __ldg(a.w + t * a.k + j) * __ldg(a.dw + t * a.k + j);
                any = true;
            }
        }
        __syncwarp();
        D = sel_sum<W>(D);
#pragma unroll
        for (int o = W / 2; o; o >>= 1) any |= __shfl_xor_sync(0xffffffffu, any, o);
        float x[V];
        auto place = [&](int i) { return VEC ? 4 * (gl + W * (i >> 2)) + (i & 3) : gl + W * i; };
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        // (a token without picks has no gradient, and its logits may be anything)
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                if (any && place(i) < a.E) {
                    if (a.bf16) sel_load4<true>(static_cast<const __nv_bfloat16*>(a.logits) + t * a.E + place(i), x + i);
                    else sel_load4<false>(static_cast<const float*>(a.logits) + t * a.E + place(i), x + i);
                }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (any && place(i) < a.E) x[i] = sel_value(row, t * a.E + place(i));
        }
        float m = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
        m = sel_max<W>(m);
        if (m == -INFINITY) m = 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = sel_exp(x[i] - m);
            sum += x[i];
        }
        sum = sel_sum<W>(sum);
        const float f = any ? -D / sum : 0.f;
        if (live) {
#pragma unroll
            for (int i = 0; i < V; i += VEC ? 4 : 1) {
                if (place(i) >= a.E) continue;
                const long long at = t * a.E + place(i);
                if constexpr (VEC) {
                    float d[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) d[q] = any ? x[i + q] * f : 0.f;
                    if (a.out_bf16) {
                        __nv_bfloat162 lo = __floats2bfloat162_rn(d[0], d[1]), hi = __floats2bfloat162_rn(d[2], d[3]);
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dlogits) + at) =
                            make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
                    } else {
                        float4* out = reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + at);
                        const float4 was = a.accumulate ? *out : make_float4(0.f, 0.f, 0.f, 0.f);
                        *out = make_float4(was.x + d[0], was.y + d[1], was.z + d[2], was.w + d[3]);
                    }
                } else {
                    const float d = any ? x[i] * f : 0.f;
                    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.dlogits)[at] = __float2bfloat16(d);
                    else static_cast<float*>(a.dlogits)[at] = (a.accumulate ? static_cast<float*>(a.dlogits)[at] : 0.f) + d;
                }
            }
        }
        __syncwarp();   // the row's values are ordered before the picks' that replace them
        for (int j = gl; live && j < a.k; j += W) {
            const int e = __ldg(a.idx + t * a.k + j);
            if ((unsigned)e >= (unsigned)a.E) continue;
            const float d = __ldg(a.w + t * a.k + j) * __ldg(a.dw + t * a.k + j);
            const long long at = t * a.E + e;
            if (a.accumulate) static_cast<float*>(a.dlogits)[at] += d;
            else if (a.out_bf16) static_cast<__nv_bfloat16*>(a.dlogits)[at] = __float2bfloat16(d + sel_exp(sel_value(row, at) - m) * f);
            else static_cast<float*>(a.dlogits)[at] = d + sel_exp(sel_value(row, at) - m) * f;
        }
        __syncwarp();
    }
}

// b[e] += rate sign(total / E - n[e]), n[e] the counts of all segments; whole numbers throughout
__global__ void __launch_bounds__(1024) select_bias_kernel(const int* __restrict__ counts, int B, int E, float* bias, float rate) {
    grid_dep_wait();
    __shared__ long long part[32];
    __shared__ long long n[kMaxExperts];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < E; e += 1024) n[e] = 0;
    __syncthreads();
    long long sum = 0;
    // threads of a column share it out where experts are few
    const int each = 1024 / E, share = threadIdx.x / E, e = threadIdx.x % E;
    if (share < each) {
        for (int b = share; b < B; b += each) sum += __ldg(counts + (long long)b * E + e);
        atomicAdd(reinterpret_cast<unsigned long long*>(n + e), (unsigned long long)sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    long long total = part[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (threadIdx.x < E) {
        const long long d = total - n[threadIdx.x] * E;
        if (d) bias[threadIdx.x] += d > 0 ? rate : -rate;
    }
}

// ---- launches --------------------------------------------------------------------------------------------------
cudaError_t launch_select_fwd(cudaStream_t st, SelectArgs a, int num_sms) {
    if (a.T == 0) return cudaSuccess;
    a.gs = a.E / a.G;
    const int bits = log2_of(a.E);
    a.low = (1u << bits) - 1u;
    a.quantum = (float)(1 << bits) * 1.1920929e-7f;   // what the last bits hold, relative to c
    // Values a lane: 4 or 8 and a whole warp where there are few tokens (2400 x 128 3.7 us, 4.3 with 16 values and 8 lanes; 2400 x
    // 256 in 8 groups 8.5 and 9.6; from 4800 on it is the other way round), 16 otherwise; more where groups do not fit 32 lanes.
    int V = 0, W = 32, lanes = 32;
    a.few = a.T <= 16 * num_sms;
    for (int v : {4, 8, 16, 32, 64}) {
        if (v < 16 && !a.few) continue;
        lanes = pow2_at_least((a.gs + v - 1) / v);
        if ((long long)a.G * lanes > 32) continue;
        V = v;
        W = v == 16 ? pow2_at_least(a.G * lanes) : 32;
        break;
    }
    if (V == 0) return cudaErrorInvalidValue;
    if (V != 16 && a.G == 1) lanes = 32;   // (the whole warp's)
    a.lpg_log2 = log2_of(lanes);
    if (a.gs % 4 != 0) return select_kind<kSelOdd>(st, a, W, V, num_sms);
    return a.gs == V * lanes && a.G * lanes == W ? select_kind<kSelFull>(st, a, W, V, num_sms) : select_kind<kSelVec>(st, a, W, V, num_sms);
}

template <int W, int V>
static cudaError_t dense_c(cudaStream_t st, const SelectGradArgs& a, int num_sms) {
    const unsigned grid = sel_grid(a.T, 8 * (32 / W), V == 16 ? 4 : 2, num_sms);
    return a.E % 4 == 0 ? launch_pdl(select_bwd_dense_kernel<W, V, true>, grid, 256, 0, st, a)
                        : launch_pdl(select_bwd_dense_kernel<W, V, false>, grid, 256, 0, st, a);
}

cudaError_t launch_select_bwd(cudaStream_t st, SelectGradArgs a, int num_sms) {
    if (a.T == 0) return cudaSuccess;
    if (!a.sigmoid && !a.renorm) {
        if (a.E <= 16) return dense_c<1, 16>(st, a, num_sms);
        if (a.E <= 32) return dense_c<2, 16>(st, a, num_sms);
        if (a.E <= 64) return dense_c<4, 16>(st, a, num_sms);
        if (a.E <= 128) return dense_c<8, 16>(st, a, num_sms);
        if (a.E <= 256) return dense_c<16, 16>(st, a, num_sms);
        if (a.E <= 512) return dense_c<32, 16>(st, a, num_sms);
        return dense_c<32, 32>(st, a, num_sms);
    }
    if (a.accumulate) {
        const int per = 8 * (32 / pow2_at_least(a.k));
        return launch_pdl(select_bwd_add_kernel, (unsigned)((a.T + per - 1) / per), 256, 0, st, a);
    }
    // Tokens of a tile: 4 (bf16: 8), so that a tile is a multiple of 16 bytes; as many as give each lane a pick; where rows are so
    // short that this is under 2 KB, more, while each SM has eight tiles.
    const int es = a.out_bf16 ? 2 : 4;
    a.tile = std::max(a.out_bf16 ? 8 : 4, 32 / pow2_at_least(a.k));
    while (a.tile > (a.out_bf16 ? 8 : 4) && a.tile * a.E * es > 8192) a.tile /= 2;
    while (a.tile * a.E * es < 2048 && a.tile < 64 && (long long)a.T >= 16LL * a.tile * num_sms) a.tile *= 2;
    const size_t smem = (size_t)kSparseWarps * 2 * a.tile * (a.E * es + 4 * a.k);   // at most 136 KB
    auto kern = a.out_bf16 ? select_bwd_sparse_kernel<true> : select_bwd_sparse_kernel<false>;
    static PerDevice<int> allowed[2];
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = allowed[a.out_bf16].get(dev, &done, [&](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 140 * 1024);
    });
    if (e != cudaSuccess) return e;
    const int blocks_sm = (int)std::max<size_t>(1, std::min<size_t>(8, 200 * 1024 / smem));
    return launch_pdl(kern, sel_grid(a.T, a.tile * kSparseWarps, blocks_sm, num_sms), 32 * kSparseWarps, smem, st, a);
}

cudaError_t launch_select_bias(cudaStream_t st, const int* counts, int B, int E, float* bias, float rate) {
    return launch_pdl(select_bias_kernel, 1, 1024, 0, st, counts, B, E, bias, rate);
}

}  // namespace moe
