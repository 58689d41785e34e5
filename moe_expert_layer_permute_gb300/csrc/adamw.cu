// adamw.cu - one AdamW step over many tensors at once, states in 32 bits or in 8, and the norm of many gradients.
//
//   g' = scale g;  m' = b1 m + (1 - b1) g';  v' = b2 v + (1 - b2) g'^2
//   p' = p - lr (m' / (1 - b1^t) / (sqrt(v' / (1 - b2^t)) + eps) + decay p)
//
// In 8 bits m and r = sqrt(v) are E4M3 codes times one fp32 scale for each 256 values of a tensor, x = code scale with
// scale = max|x| / 448.  Rounded to nearest such a state would stand still: with b2 = 0.999 a step moves v by a
// thousandth, and half a code's step is 3 to 6 %.  So x goes up to the next code with the probability of its distance to
// the one below, by 16 bits of a hash of the seed, the tensor's number and the value's: exact in the mean.  r's codes are
// at least the smallest, so that no v that a gradient has touched becomes 0 beside an m that has not.
// What that leaves: at steady state v is 1.05 times the 32-bit state's in the mean, its root 17 % off (rms, of itself) and m 8 %
// (of its rms), at any level of the gradients (4096 values, 3000 steps at each of three levels); with the same bits at every step
// v is 2.3 times too large and its root 70 % off.
//
// Bound by memory: 28 bytes a value (fp32 gradients and states), 14 (bf16 gradients, 8-bit states), 2 more for the
// bf16 copy.  604 M values with the copy: fp32 2.8 ms (6.5 TB/s, 0.97 of a copy's rate), 8 bits 1.71 ms (5.7 TB/s, 0.85).  A warp takes 256 neighbouring values at a time, 4 a lane in two groups, so that every access is a row of
// whole sectors and a block of 8-bit states is one warp's: its largest value is one reduction, and no warp waits for
// another.  The tensors' addresses come as the launch's arguments, up to 384 tensors of any sizes a launch (by a table in
// memory each call would wait for a copy).
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kAdamWarps = kListWarps;
constexpr int kAdamUnit = kListUnit;   // and values of a block of 8-bit states
// Blocks an SM.  In 8 bits a value is some 85 instructions and 14 to 18 bytes, so that issue slots and memory are both near
// their ends (74 % and 85 %) and more warps cover more of the wait: with 4 blocks (64 registers a thread) 604 M values take
// 6 % longer than with 5, with 6 (spills) 3 %.
template <bool EIGHT>
constexpr int adam_blocks_sm() { return EIGHT ? 5 : 4; }
constexpr int kNormChunk = 4;      // neighbouring units of a warp's, all under way at once (a block's 32 stand together)
constexpr int kNormSteps = 16;     // units that a lane adds up in 32 bits

template <int MOST>
struct ListArgs {
    ListTensor tensor[MOST];
    int start[MOST + 1];           // units before each tensor
    int count;
};
// the tensor of unit u, which is at `at` or behind it
template <int MOST>
__device__ __forceinline__ int list_find(const ListArgs<MOST>& a, int at, int u) {
    if (u < a.start[at + 1]) return at;
    int lo = at + 1, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (u >= a.start[mid]) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// four fp32 or bf16 values at place i, which a warp whose unit is whole (ALL) takes in one access; `left` of them are
// there
template <bool ALL>
__device__ __forceinline__ void list_load4(float* x, const void* p, bool bf16, long long i, int left) {
    if (ALL) {
        if (bf16) {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
            x[0] = __uint_as_float(v.x << 16);
            x[1] = __uint_as_float(v.x & 0xffff0000u);
            x[2] = __uint_as_float(v.y << 16);
            x[3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q] = 0.f;
            if (q < left) x[q] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i + q]) : static_cast<const float*>(p)[i + q];
        }
    }
}
template <bool ALL>
__device__ __forceinline__ void list_store4(float* p, const float* x, long long i, int left) {
    if (ALL) {
        *reinterpret_cast<float4*>(p + i) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < left) p[i + q] = x[q];
    }
}
template <bool ALL>
__device__ __forceinline__ void list_store4(__nv_bfloat16* p, const float* x, long long i, int left) {
    if (ALL) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2*>(p + i) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < left) p[i + q] = __float2bfloat16(x[q]);
    }
}
template <bool ALL>
__device__ __forceinline__ uint32_t list_load_codes(const void* p, long long i, int left) {
    const uint8_t* c = static_cast<const uint8_t*>(p) + i;
    if (ALL) return *reinterpret_cast<const uint32_t*>(c);
    uint32_t v = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (q < left) v |= (uint32_t)c[q] << (8 * q);
    return v;
}
template <bool ALL>
__device__ __forceinline__ void list_store_codes(void* p, uint32_t v, long long i, int left) {
    uint8_t* c = static_cast<uint8_t*>(p) + i;
    if (ALL) {
        *reinterpret_cast<uint32_t*>(c) = v;
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < left) c[q] = (uint8_t)(v >> (8 * q));
    }
}
// four E4M3 codes times a scale, one rounding each
__device__ __forceinline__ void decode4(float* x, uint32_t codes, float scale) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> (16 * h)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        x[2 * h] = __fmul_rn(f.x, scale);
        x[2 * h + 1] = __fmul_rn(f.y, scale);
    }
}
// 32 random bits of a value's number: C. Wellons's published mixing of 32 bits (2018; xor-shifts of 16, 15 and 16, and two
// multipliers of the least bias that a search found) over its place in a Weyl sequence of the golden ratio
__device__ __forceinline__ uint32_t adam_noise(uint32_t place, uint32_t key) {
    uint32_t h = place * 0x9E3779B1u + key;
    h = (h ^ (h >> 16)) * 0x7FEB352Du;
    h = (h ^ (h >> 15)) * 0x846CA68Bu;
    return h ^ (h >> 16);
}
// |x| up, from 0 to 448 and a rounding, to a code: times 2^-120 the codes are the leading bits of the fp32 form (those
// below 2^-6 the leading bits of numbers without an exponent), and a carry into them is the step up.  noise4: 16 random
// bits, times 16; 8 is the middle of what they leave open.
__device__ __forceinline__ uint32_t encode(float x, float up, uint32_t noise4) {
    const float y = __fmul_rn(__fmul_rn(fabsf(x), up), 7.52316384526264e-37f);   // 2^-120
    return min((__float_as_uint(y) + noise4 + 8u) >> 20, 126u);
}
// the low bytes of four
__device__ __forceinline__ uint32_t bytes4(const uint32_t* c) {
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
// the larger of most and |x|, NaN if either is
__device__ __forceinline__ float max_abs(float most, float x) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(most), "f"(x));
    return r;
}
// what the codes of a block are scaled by: its largest value's bits -> 448 / it (0: none, or not finite) and the scale
__device__ __forceinline__ float block_scale(uint32_t most, float* scale) {
    float s = __uint_as_float(most);
    if (s < 1e-35f) s = 0.f;
    *scale = __fmul_rn(s, 1.f / 448.f);
    return s > 0.f ? __fmul_rn(__frcp_rn(s), 448.f) : 0.f;
}

template <int MOST, bool EIGHT>
__global__ void __launch_bounds__(32 * kAdamWarps, adam_blocks_sm<EIGHT>()) adamw_kernel(const __grid_constant__ ListArgs<MOST> list, const AdamArgs a) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f;
    if (!(fabsf(gs) < INFINITY)) return;   // no step
    const float lr = a.lr_at ? __ldg(a.lr_at) : a.lr;
    float fix1 = a.fix1, fix2 = a.fix2;
    uint32_t seed = a.seed;
    if (a.step_at) {
        // 1 - b^t = -expm1(t ln b), t ln b to 2^-24 of itself, and so its result
        const int number = __ldg(a.step_at);
        if (number < 1) return;   // no step either: nothing corrects a mean of no gradients
        const float t = (float)number;
        fix1 = 1.f / -expm1f(t * a.log_b1);
        fix2 = rsqrtf(-expm1f(t * a.log_b2));
        seed += (uint32_t)number;
    }
    const int units = list.start[list.count], stride = gridDim.x * kAdamWarps;
    int u = blockIdx.x * kAdamWarps + (threadIdx.x >> 5);
    if (u >= units) return;
    const float step_size = -lr;
    auto unit = [&](const ListTensor& t, long long block, auto all) {
        constexpr bool ALL = decltype(all)::value;
        const long long first = block * kAdamUnit + 4 * lane;
        float p[8], g[8], m[8], v[8];
        int left[2] = {4, 4};
        [[maybe_unused]] float ms = 0.f, vs = 0.f;
        [[maybe_unused]] uint32_t mc[2], vc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long i = first + 128 * h;
            if (!ALL) left[h] = (int)max(min(t.n - i, 4ll), 0ll);
            list_load4<ALL>(g + 4 * h, t.g, t.g_bf16, i, left[h]);
            list_load4<ALL>(p + 4 * h, t.p, false, i, left[h]);
            if constexpr (EIGHT) {
                mc[h] = list_load_codes<ALL>(t.m, i, left[h]);
                vc[h] = list_load_codes<ALL>(t.v, i, left[h]);
            } else {
                list_load4<ALL>(m + 4 * h, t.m, false, i, left[h]);
                list_load4<ALL>(v + 4 * h, t.v, false, i, left[h]);
            }
        }
        if constexpr (EIGHT) {
            ms = t.m_scale[block];
            vs = t.v_scale[block];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                decode4(m + 4 * h, mc[h], ms);
                decode4(v + 4 * h, vc[h], vs);
            }
        }
        // Roundings as they stand in the formulas, none of them fused: one more or less in a million moves a code, and that
        // code's value the next step by a tenth.  The root is the library's, rounded to nearest (a Newton step on an approximate
        // one and the library's beyond its range took 1707 us instead of 1708 for 604 M values in 8 bits, 3170 instead of 3182 in 32).
        [[maybe_unused]] float most_m = 0.f, root[8];
        float most_v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = __fmul_rn(g[i], gs);
            if constexpr (EIGHT) v[i] = __fmul_rn(v[i], v[i]);
            m[i] = __fadd_rn(__fmul_rn(m[i], a.b1), __fmul_rn(x, a.c1));
            v[i] = __fadd_rn(__fmul_rn(v[i], a.b2), __fmul_rn(__fmul_rn(x, x), a.c2));
            root[i] = __fsqrt_rn(v[i]);
            most_v = max_abs(most_v, v[i]);
            if constexpr (EIGHT) most_m = max_abs(most_m, m[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float step = (m[i] * fix1) * rcp_approx(fmaf(root[i], fix2, a.eps));
            p[i] = fmaf(step_size, fmaf(a.decay, p[i], step), p[i]);
        }
        if constexpr (EIGHT) {
            const uint32_t mm = __reduce_max_sync(0xffffffffu, __float_as_uint(most_m));   // (NaN is above infinity)
            const uint32_t vm = __reduce_max_sync(0xffffffffu, __float_as_uint(most_v));
            const float mu = block_scale(mm, &ms), vu = block_scale(__float_as_uint(__fsqrt_rn(__uint_as_float(vm))), &vs);
            const uint32_t key = seed + (uint32_t)(t.ordinal + 1) * 0x85EBCA77u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t place = (uint32_t)(first + 128 * h);
                uint32_t cm[4], cv[4], sign[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t noise = adam_noise(place + q, key);
                    sign[q] = __float_as_uint(m[4 * h + q]) >> 24;
                    cm[q] = encode(m[4 * h + q], mu, (noise << 4) & 0xffff0u);
                    cv[q] = max(encode(root[4 * h + q], vu, (noise >> 12) & 0xffff0u), 1u);
                }
                list_store_codes<ALL>(t.m, mu > 0.f ? bytes4(cm) | (bytes4(sign) & 0x80808080u) : 0u, first + 128 * h, left[h]);
                list_store_codes<ALL>(t.v, vu > 0.f ? bytes4(cv) : 0u, first + 128 * h, left[h]);
            }
            if (lane == 0) {
                t.m_scale[block] = ms;
                t.v_scale[block] = vs;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long i = first + 128 * h;
            list_store4<ALL>(t.p, p + 4 * h, i, left[h]);
            if constexpr (!EIGHT) {
                list_store4<ALL>(static_cast<float*>(t.m), m + 4 * h, i, left[h]);
                list_store4<ALL>(static_cast<float*>(t.v), v + 4 * h, i, left[h]);
            }
            if (t.copy) list_store4<ALL>(t.copy, p + 4 * h, i, left[h]);
        }
    };
    for (int at = 0; u < units; u += stride) {
        at = list_find(list, at, u);
        const ListTensor& t = list.tensor[at];
        const long long block = u - list.start[at];
        if ((block + 1) * kAdamUnit <= t.n) unit(t, block, std::true_type{});
        else unit(t, block, std::false_type{});
    }
}

// Sum of squares: a lane adds up kNormSteps units in 32 bits, those sums and all others in 64.  A block's sum goes to
// partial[its number in all launches]; the block that finishes last adds them in their order, so that the result does
// not depend on who came when.
template <int MOST>
__global__ void __launch_bounds__(32 * kAdamWarps, 4) norm_kernel(const __grid_constant__ ListArgs<MOST> list, const NormArgs a) {
    grid_dep_wait();
    __shared__ double part[kAdamWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = list.start[list.count], stride = gridDim.x * kAdamWarps;
    double sum = 0.0;
    for (int at = 0, c = blockIdx.x * kAdamWarps * kNormChunk + warp; c < units; ) {
        float s0 = 0.f, s1 = 0.f;
        for (int k = 0; k < kNormSteps / kNormChunk && c < units; ++k, c += stride * kNormChunk) {
#pragma unroll
            for (int j = 0; j < kNormChunk; ++j) {
                const int u = c + j * kAdamWarps;
                if (u >= units) break;
                at = list_find(list, at, u);
                const ListTensor& t = list.tensor[at];
                const long long first = (long long)(u - list.start[at]) * kAdamUnit + 4 * lane;
                float g[8];
                const bool all = (u - list.start[at] + 1ll) * kAdamUnit <= t.n;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (all) list_load4<true>(g + 4 * h, t.g, t.g_bf16, first + 128 * h, 4);
                    else list_load4<false>(g + 4 * h, t.g, t.g_bf16, first + 128 * h, (int)max(min(t.n - first - 128 * h, 4ll), 0ll));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s0 = fmaf(g[i], g[i], s0);
                    s1 = fmaf(g[4 + i], g[4 + i], s1);
                }
            }
        }
        sum += (double)(s0 + s1);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    sum = part[lane % kAdamWarps];
#pragma unroll
    for (int o = kAdamWarps / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    bool last = false;
    if (lane == 0) {
        a.partial[a.first_block + blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(a.ticket, 1) == a.blocks - 1;
    }
    last = __shfl_sync(0xffffffffu, (int)last, 0);
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int i = lane; i < a.blocks; i += 32) sum += __ldcg(a.partial + i);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        // the root in 32 bits where the sum has its place there
        const float norm = sum > 1e-30 && sum < 1e38 ? sqrtf((float)sum) : (float)sqrt(sum);
        a.out[0] = norm;
        // not a number where the norm is none or infinite, which a step takes as no step
        a.out[1] = !(norm < INFINITY) ? NAN : a.most > 0.f && norm > a.most ? a.most / norm : 1.f;
        *a.ticket = 0;
    }
}

// ---- launches --------------------------------------------------------------------------------------------------
template <int MOST>
static void list_args(ListArgs<MOST>* a, const ListTensor* t, int count) {
    a->count = count;
    memcpy(a->tensor, t, count * sizeof(ListTensor));
    int at = 0;
    for (int i = 0; i < count; ++i) {
        a->start[i] = at;
        at += (int)((t[i].n + kAdamUnit - 1) / kAdamUnit);
    }
    a->start[count] = at;
}
// (without the copies that passing the lists by value would make)
template <int MOST, typename A>
static cudaError_t list_launch(cudaStream_t st, void (*kern)(ListArgs<MOST>, A), int blocks, const ListArgs<MOST>& list, const A& a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * kAdamWarps);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<ListArgs<MOST>*>(&list), const_cast<A*>(&a)};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kern), args);
}

template <int MOST>
static cudaError_t adamw_n(cudaStream_t st, const ListTensor* t, int count, bool eight, const AdamArgs& a, int num_sms) {
    ListArgs<MOST> list;
    list_args(&list, t, count);
    const int most = (eight ? adam_blocks_sm<true>() : adam_blocks_sm<false>()) * num_sms;
    const int blocks = std::max(1, std::min((list.start[count] + kAdamWarps - 1) / kAdamWarps, most));
    return list_launch(st, eight ? adamw_kernel<MOST, true> : adamw_kernel<MOST, false>, blocks, list, a);
}
// (a launch with few tensors has fewer bytes of arguments)
cudaError_t launch_adamw(cudaStream_t st, const ListTensor* t, int count, bool eight, const AdamArgs& a, int num_sms) {
    if (count <= 8) return adamw_n<8>(st, t, count, eight, a, num_sms);
    if (count <= 48) return adamw_n<48>(st, t, count, eight, a, num_sms);
    return adamw_n<kListMost>(st, t, count, eight, a, num_sms);
}

int norm_blocks(const ListTensor* t, int count, int num_sms) {
    long long units = 0;
    for (int i = 0; i < count; ++i) units += list_units(t[i].n);
    return norm_blocks_of(units, num_sms);
}
template <int MOST>
static cudaError_t norm_n(cudaStream_t st, const ListTensor* t, int count, const NormArgs& a, int num_sms) {
    ListArgs<MOST> list;
    list_args(&list, t, count);
    return list_launch(st, norm_kernel<MOST>, norm_blocks(t, count, num_sms), list, a);
}
cudaError_t launch_norm(cudaStream_t st, const ListTensor* t, int count, const NormArgs& a, int num_sms) {
    if (count <= 8) return norm_n<8>(st, t, count, a, num_sms);
    if (count <= 48) return norm_n<48>(st, t, count, a, num_sms);
    return norm_n<kListMost>(st, t, count, a, num_sms);
}

}  // namespace moe
