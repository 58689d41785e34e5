// select.cu - routing by scores: each token's k experts by the scores of all of them, with a bias that only the
// choice sees and with groups of experts, the weights' gradient, and the step that moves the bias.
//
//   s = softmax(l) or sigmoid(l);  c = s + b;  an expert with l = -inf or b = -inf is excluded
//   group g: the sum of its `rank` largest c; the `kept` groups with the largest sums stay
//   picks: the k largest c of what stays, descending;  w_j = scale s_j (/ sum of the picks' s)
//
// Picks have to be the same wherever and however often they are computed, so c and the sums are compared in 64 bits
// (without a bias the logits themselves, whose order is that of the scores), equal ones by their index.  Sums of a score
// and a bias that lie within fp32's error of each other come up in about one token of a thousand (16,384 x 256), so
// the forward works on fp32 and knows its error: where two neighbours of the result, or two groups at the border, are
// nearer than that, the token alone is gone through again (select_again below).
//
// Forward.  W lanes hold one token's logits in registers, V each (V = 16 in batches of many tokens: 32 / W tokens
// share a warp's instructions; 4 or 8 where tokens are few and latency counts), a group of experts in lanes of its
// own.  A value is a 32-bit key, c's bits in an order that compares as unsigned, whose last bits hold E - e: keys
// are unlike, so one maximum finds value and index, and the largest key below the last pick p is
// p + max_i(key_i - p) modulo 2^32, two instructions a value (three and a half with a mark and a search).  What the
// index takes from c (7 bits at 128 experts) is part of the error above; it is small where the numbers are, so c is taken
// relative to the largest bias and then to the row's largest c.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "per_device.h"

namespace moe {

constexpr int kSelWarps = 4;

__device__ __forceinline__ float sel_value(const SelectArgs& a, long long i) {
    return a.bf16 ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(a.logits) + i))
                  : __ldg(static_cast<const float*>(a.logits) + i);
}
// four of them, 16-byte (bf16: 8-byte) aligned
template <bool BF>
__device__ __forceinline__ void sel_load4(const void* p, float* x) {
    if constexpr (BF) {
        const uint2 v = __ldg(static_cast<const uint2*>(p));
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
        const float4 v = __ldg(static_cast<const float4*>(p));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
}
template <bool BF>
__device__ __forceinline__ float sel_load(const void* p) {
    if constexpr (BF) return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p)));
    else return __ldg(static_cast<const float*>(p));
}
// A float's order as an unsigned number: -0 is 0, NaN above everything, -inf 0x007fffff
__device__ __forceinline__ uint32_t sel_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);   // (-0 + 0 is +0, a sum of any NaN the one NaN 0x7fffffff)
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float sel_unkey(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t sel_key64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return v == v ? u ^ ((uint64_t)((long long)u >> 63) | 0x8000000000000000ull) : ~0ull;
}
__device__ __forceinline__ double sel_unkey64(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? k ^ 0x8000000000000000ull : ~k));
}
__device__ __forceinline__ float sel_exp(float x) { return exp2_approx(x * 1.442695041f); }
__device__ __forceinline__ float sel_sigmoid(float x) { return rcp_approx(1.f + sel_exp(-x)); }   // (0 for an infinite power)

// How far an fp32 score may be from the exact one where it is at most `most`.  The power is off by 2^-22 relative, its
// argument z (times log2 e) by 2^-24 of it, a quotient by 2^-23.
//   sigmoid: s (1 - s) (2^-22 + 2^-23 |z|) + 2^-23 s, at most 3e-7, and for a small s, -z up to 88, 1.1e-5 s
//   softmax: s (2^-22 + 2^-23 (-ln s)) and the sum's error, some 2^-21 with its exponentials'; s (-ln s) is at most 0.37
__device__ __forceinline__ float sel_error(bool sigmoid, float most) {
    const float s = fminf(fmaxf(most, 1e-37f), 1.f);
    return sigmoid ? fminf(3e-7f, 1.1e-5f * s) : 9e-7f * s + fminf(4.5e-8f, 1.1e-5f * s);
}
constexpr float kSelSum = 1.2e-7f;   // of a sum's size: a rounding of it, and one of its bias less the largest

template <int W>
__device__ __forceinline__ float sel_max(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int W>
__device__ __forceinline__ uint32_t sel_max(uint32_t v) {
    if constexpr (W == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int W>
__device__ __forceinline__ float sel_sum(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// sum over segments of n lanes, n a power of two
__device__ __forceinline__ float sel_segment_sum(float v, int n) {
    for (int o = n >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float sel_segment_max(float v, int n) {
    for (int o = n >> 1; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// ---- one token again, exactly, by a whole warp ---------------------------------------------------------------
// A pick as the forward keeps it: 0 for none, else bits of a key, the last of which hold low - e.
__device__ __forceinline__ uint32_t sel_pick(int e, uint32_t low) { return 0xff000000u | (low - (uint32_t)e); }

// e^y in 64 bits, to some 2^-52, for y in [-708, 708] (beyond it the ends' values): 2^n times the power series of what is
// left of y, at most ln 2 / 2, whose term 14 is under 2^-57.  The code that follows runs for a few tokens of a thousand
// and mostly waits for its own instructions, so it is kept short and out of line, its loops rolled (with the library's
// exponential and quotient and the loops unrolled 16,384 x 256 in 8 groups took 19.5 us).
__device__ __noinline__ double sel_exp64(double y) {
    if (y > 708.0) y = 708.0;
    if (y < -708.0) y = -708.0;   // (a NaN stays)
    const double n = rint(y * 1.4426950408889634);
    const double r = fma(n, -2.3190468138462996e-17, fma(n, -0.6931471805599453, y));
    double p = 1.0 / 6227020800.0, f = 1.0 / 479001600.0;
    p = fma(p, r, f);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return p * __hiloint2double((__double2int_rn(n) + 1023) << 20, 0);
}
// The score of logit x; a softmax's with the row's largest logit and 1 / sum.
__device__ __forceinline__ double sel_score64(const SelectArgs& a, float x, double row_max, double inv_sum) {
    const double z = sel_exp64(a.sigmoid ? -(double)x : (double)x - row_max);
    if (!a.sigmoid) return z * inv_sum;
    // 1 / (1 + z): from fp32's, or its exponent alone, by Newton's steps, each of which doubles the digits
    const double d = 1.0 + z;
    double q = d < 1e30 ? (double)rcp_approx((float)d) : 1.0 / d;
#pragma unroll
    for (int i = 0; i < 2; ++i) q = fma(q, fma(-d, q, 1.0), q);
    return q;
}

struct SelRoom {              // a warp's shared memory
    uint64_t sorted[32];
    int candidate[32];
};
struct SelToken {             // what the forward found out about a token
    float top;                // its largest c, less the largest bias
    float max, inv;           // of the softmax: the largest logit and 1 / sum
    uint32_t groups;          // bits of those that stay; 0: not known
};

// How far two sums may come nearer to each other than they are in fp32: scores of at most `most`, roundings of sums, biases
// and distances from `top`, of which d is the larger; `quantum` is what the index has taken from d, if anything.
__device__ __forceinline__ float sel_margin(const SelectArgs& a, float top, float d, float most, float quantum) {
    return 2.f * sel_error(a.sigmoid, most) + 2.f * kSelSum * (fabsf(top) + d) + (quantum + kSelSum) * d;
}

// Every expert in 64 bits, their groups too: k rounds of the largest that is left.
__device__ __noinline__ void select_all(const SelectArgs& a, long long t, uint32_t low, uint32_t* picks) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const bool scores = a.bias || a.G > 1;
    // keys of expert lane + 32 i (0: excluded, or taken)
    uint64_t key[32];
    const int rows = (a.E + 31) >> 5;
    double top = -INFINITY, sum = 0.0;
    if (!a.sigmoid && scores) {
        bool nan = false;
#pragma unroll 1
        for (int i = 0; i < rows; ++i)
            if (lane + 32 * i < a.E) {
                const float x = sel_value(a, t * a.E + lane + 32 * i);
                nan |= isnan(x);
                top = fmax(top, (double)x);
            }
#pragma unroll 1
        for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(all, top, o));
        if (__any_sync(all, nan)) top = NAN;
#pragma unroll 1
        for (int i = 0; i < rows; ++i)
            if (lane + 32 * i < a.E) sum += sel_exp64((double)sel_value(a, t * a.E + lane + 32 * i) - top);
#pragma unroll 1
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(all, sum, o);
    }
    const double inv = 1.0 / sum;
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0;
        if (e >= a.E) continue;
        const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) : 0.f;
        if (x == -INFINITY || b == -INFINITY) continue;
        double c = (double)x;
        if (scores) c = sel_score64(a, x, top, inv) + (double)b;
        key[i] = sel_key64(c);
    }
    if (a.G > 1) {
        uint64_t value = 0;   // of group `lane`
#pragma unroll 1
        for (int g = 0; g < a.G; ++g) {
            uint64_t m1 = 0, m2 = 0;
#pragma unroll 1
            for (int i = 0; i < rows; ++i) {
                const int e = lane + 32 * i;
                if (e < g * a.gs || e >= (g + 1) * a.gs) continue;
                const uint64_t v = key[i];
                m2 = max(m2, min(m1, v));
                m1 = max(m1, v);
            }
#pragma unroll 1
            for (int o = 16; o; o >>= 1) {
                const uint64_t o1 = __shfl_xor_sync(all, m1, o), o2 = __shfl_xor_sync(all, m2, o);
                m2 = max(max(m2, o2), min(m1, o1));
                m1 = max(m1, o1);
            }
            if (a.rank == 2 && m2) m1 = sel_key64(sel_unkey64(m1) + sel_unkey64(m2));
            if (lane == g) value = m1;
        }
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < a.G; ++g) {
            const uint64_t other = __shfl_sync(all, value, g);
            rank += other > value || (other == value && g < lane);
        }
        const uint32_t kept = __ballot_sync(all, lane < a.G && value && rank < a.kept);
#pragma unroll 1
        for (int i = 0; i < rows; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> (e / a.gs)) & 1u)) key[i] = 0;
        }
    }
    if (!a.bias && a.G > 1)
#pragma unroll 1
        for (int i = 0; i < rows; ++i)
            if (key[i]) key[i] = sel_key64((double)sel_value(a, t * a.E + lane + 32 * i));
#pragma unroll 1
    for (int r = 0; r < a.k; ++r) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll 1
        for (int i = 0; i < rows; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        uint64_t top_key = best;
        int e = lane + 32 * at;
#pragma unroll 1
        for (int o = 16; o; o >>= 1) {
            const uint64_t ok = __shfl_xor_sync(all, top_key, o);
            const int oe = __shfl_xor_sync(all, e, o);
            if (ok > top_key || (ok == top_key && oe < e)) {
                top_key = ok;
                e = oe;
            }
        }
        if (top_key && (e & 31) == lane) key[e >> 5] = 0;
        if (lane == 0) picks[r] = top_key ? sel_pick(e, low) : 0u;
    }
    __syncwarp();
}

// open: bit j where picks j and j + 1 are too near each other.  The candidates are those from the first such pick on, as
// far as their order is open (picks before and after them stand), and where the last pick is among them every expert
// that may be; the fp32 sums in full decide where they are far enough apart, else sums in 64 bits (a softmax's over
// its fp32 sum, whose error stands in both terms and so counts with their difference alone).  Where that is not enough
// either, or there are more than 32, or nothing is known (0), all experts are gone through.
__device__ __noinline__ void select_again(const SelectArgs& a, long long t, uint32_t open, const SelToken& token, float span,
                                          float top_bias, uint32_t low, uint32_t none, SelRoom* room, uint32_t* picks) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const bool scores = a.bias || a.G > 1;
    const float row_max = token.max, inv_sum = token.inv;
    int from = 0, n = 33;
    if (open) {
        from = __ffs(open) - 1;
        n = min(33 - __clz(open), a.k) - from;
        if (lane < n) room->candidate[lane] = (int)(low - (picks[from + lane] & low));
        if ((open >> (a.k - 1)) & 1u) {
            const uint32_t next = picks[a.k];
            const int mine = lane < a.k ? (int)(low - (picks[lane] & low)) : -1;
            // (every score is at most 1; a softmax's at most 1 / its sum)
            const float d = __uint_as_float(~next & ~low);
            const float far = d + 2.f * sel_margin(a, token.top, d, a.sigmoid ? 1.f : inv_sum, a.quantum);
#pragma unroll 1
            for (int i = 0; i < a.E && n <= 32; i += 32) {
                const int e = i + lane;
                bool in = false;
                if (e < a.E && (a.G == 1 || ((token.groups >> (e / a.gs)) & 1u))) {
                    const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) - top_bias : 0.f;
                    if (scores)
                        in = x != -INFINITY && token.top - ((a.sigmoid ? sel_sigmoid(x) : sel_exp(x - row_max) * inv_sum) + b) <= far;
                    else
                        in = (sel_key(x) & ~low) >= (next & ~low);
                }
#pragma unroll 1
                for (uint32_t votes = __ballot_sync(all, in); votes; votes &= votes - 1) {
                    const int it = i + __ffs(votes) - 1;
                    if (__any_sync(all, mine == it)) continue;
                    if (lane == 0 && n < 32) room->candidate[n] = it;
                    ++n;
                }
            }
        }
        __syncwarp();
    }
    if (n <= 32) {
        const int e = lane < n ? room->candidate[lane] : 0;
        const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) : 0.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            float s = 0.f;
            double s64 = 0.0;
            uint64_t key;
            if (!scores) {
                key = (uint64_t)sel_key(x) << 32;
            } else if (pass == 0) {
                s = a.sigmoid ? sel_sigmoid(x) : sel_exp(x - row_max) * inv_sum;
                key = (uint64_t)sel_key(s + (b - top_bias)) << 32;
            } else {
                s64 = sel_score64(a, x, (double)row_max, (double)inv_sum);
                key = sel_key64(s64 + (double)b);
            }
            if (lane >= n) key = 0;
            int rank = 0;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const uint64_t other = __shfl_sync(all, key, i);
                const int oe = __shfl_sync(all, e, i);
                rank += other > key || (other == key && oe < e);
            }
            __syncwarp();
            if (lane < n) {
                room->sorted[rank] = key;
                room->candidate[rank] = lane;
            }
            __syncwarp();
            bool near = false;
            if (scores && !(a.sigmoid && pass == 1)) {
                const int after = lane < n && rank + 1 < n ? room->candidate[rank + 1] : lane;
                const double so = __shfl_sync(all, s64, after);
                const float xo = __shfl_sync(all, x, after), bo = __shfl_sync(all, b, after);
                if (after != lane && from + rank < a.k && !(x == xo && b == bo)) {   // (equal ones are in the order of their index)
                    const uint64_t next = room->sorted[rank + 1];
                    if (pass == 0) {
                        const float c = sel_unkey((uint32_t)(key >> 32)), d = sel_unkey((uint32_t)(next >> 32));
                        near = !(c - d > 2.f * sel_error(a.sigmoid, s + span) + kSelSum * (fabsf(c) + fabsf(d)));
                    } else {
                        const double c = sel_unkey64(key), d = sel_unkey64(next);
                        near = !(c - d > 2e-6 * fabs(s64 - so) + 1e-15 * (fabs(c) + fabs(b)));
                    }
                }
            }
            if (!__any_sync(all, near)) {
                if (lane < n && from + rank < a.k) picks[from + rank] = sel_pick(e, low);
                __syncwarp();
                return;
            }
            __syncwarp();
        }
    }
    select_all(a, t, low, picks);
}

// Groups of one token that are too near each other at the border: which of the contenders stay, `slots` of them, as a mask of
// groups; from the n candidates, which hold every expert that can be among a contender's `rank` largest, their sums in 64
// bits.  0 where a softmax's sum, which has 32, leaves it open.
__device__ __noinline__ uint32_t select_groups(const SelectArgs& a, long long t, int n, int slots, float row_max, float inv_sum,
                                               const SelRoom* room) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const int e = lane < n ? room->candidate[lane] : 0, g = lane < n ? e / a.gs : -1 - lane;
    const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) : 0.f;
    const double s = sel_score64(a, x, (double)row_max, (double)inv_sum);
    const double c = s + (double)b;
    const uint64_t key = sel_key64(c);
    int place = 0;   // in its group
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint64_t other = __shfl_sync(all, key, i);
        const int oe = __shfl_sync(all, e, i), og = __shfl_sync(all, g, i);
        place += og == g && (other > key || (other == key && oe < e));
    }
    double sum = 0.0, score = 0.0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const double oc = __shfl_sync(all, c, i), os = __shfl_sync(all, s, i);
        const int og = __shfl_sync(all, g, i), op = __shfl_sync(all, place, i);
        if (og == g && op < a.rank) {
            sum += oc;
            score += os;
        }
    }
    const bool first = lane < n && place == 0;
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const double os = __shfl_sync(all, sum, i);
        const int og = __shfl_sync(all, g, i);
        const bool of = __shfl_sync(all, (int)first, i);
        rank += of && (os > sum || (os == sum && og < g));
    }
    bool near = false;
    if (!a.sigmoid)
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const double os = __shfl_sync(all, sum, i), oc = __shfl_sync(all, score, i);
            const bool stays = __shfl_sync(all, (int)(first && rank < slots), i);
            near |= first && rank >= slots && stays && !(os - sum > 2e-6 * fabs(oc - score) + 1e-15 * (fabs(os) + 1.0));
        }
    const uint32_t mask = __reduce_or_sync(all, first && rank < slots ? 1u << g : 0u);
    return __any_sync(all, near) ? 0u : mask;
}

// ---- forward ---------------------------------------------------------------------------------------------------
// keys that a lane keeps in order: the k picks of a token fall on its W lanes, and a lane that has given all it kept looks
// through its V keys again, which the whole warp waits for
template <int W, int V>
constexpr int sel_kept() { return W == 32 && V <= 16 ? 2 : W >= 16 ? 3 : 4; }

template <int W, int V, bool VEC>
__global__ void __launch_bounds__(32 * kSelWarps, V <= 16 ? 8 : V == 32 ? 4 : 2) select_fwd_kernel(const SelectArgs a) {
    grid_dep_wait();
    constexpr int NT = 32 / W;   // tokens of a warp
    extern __shared__ __align__(16) float sel_shared[];
    __shared__ SelRoom rooms[kSelWarps];
    __shared__ SelToken tokens[kSelWarps][32];
    __shared__ float ends[2 * kSelWarps];
    const unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane % W;
    const int lpg = 1 << a.lpg_log2, group = gl >> a.lpg_log2, lp = gl & (lpg - 1);
    const uint32_t low = a.low;
    const bool scores = a.bias || a.G > 1;                 // c is not the logit
    const bool row = !a.sigmoid && (scores || !a.renorm);  // the softmax's sum is needed
    const uint32_t none = scores ? 0x80800000u : 0x00800000u;   // keys below it are no expert's
    float* biases = sel_shared;                            // less the largest
    uint32_t* picks = reinterpret_cast<uint32_t*>(sel_shared + (a.bias ? (a.E + 3) / 4 * 4 : 0)) + warp * a.batch * (a.k + 1);
    int kp = 1;                                            // lanes of a token where lanes take one pick each
    while (kp < a.k) kp *= 2;
    const int per = 32 / kp;

    float span = 0.f, top_bias = 0.f;                      // of the finite biases
    if (a.bias) {
        float hi = -INFINITY, lo = INFINITY;
        for (int e = threadIdx.x; e < a.E; e += 32 * kSelWarps) {
            const float b = __ldg(a.bias + e);
            biases[e] = b;
            if (fabsf(b) < INFINITY) {
                hi = fmaxf(hi, b);
                lo = fminf(lo, b);
            }
        }
        hi = sel_max<32>(hi);
        lo = -sel_max<32>(-lo);
        if (lane == 0) {
            ends[warp] = hi;
            ends[kSelWarps + warp] = lo;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            hi = fmaxf(hi, ends[w]);
            lo = fminf(lo, ends[kSelWarps + w]);
        }
        if (hi >= lo) {
            span = hi - lo;
            top_bias = hi;
        }
        for (int e = threadIdx.x; e < a.E; e += 32 * kSelWarps) biases[e] -= top_bias;
        __syncthreads();
    }
    auto place = [&](int i) { return VEC ? 4 * (lp + lpg * (i >> 2)) + (i & 3) : lp + lpg * i; };
    const int e0 = group * a.gs;
    const int held = group < a.G ? a.gs : 0;               // places below it hold experts
    const uint32_t code0 = low - (uint32_t)e0;
    // A warp takes `batch` tokens, NT at a time, and then all of their picks at once.
    const long long step = (long long)gridDim.x * kSelWarps * a.batch;
    for (long long first = ((long long)blockIdx.x * kSelWarps + warp) * a.batch; first < a.T; first += step) {
    for (int part = 0; part < a.batch; part += NT) {
        const int at_token = part + lane / W;
        const long long t = first + at_token;
        const bool live = t < a.T && !(a.mask && !__ldg(a.mask + t));
        const int read = live ? held : 0;
        float x[V];
        auto load = [&](auto bf) {   // (a copy of the loop for each type, so that none is chosen for each value)
            constexpr bool BF = decltype(bf)::value;
            const char* from = static_cast<const char*>(a.logits) + (t * a.E + e0 + place(0)) * (BF ? 2 : 4);
            const int stride = lpg * (BF ? 2 : 4);         // bytes between a lane's places (four times it if VEC)
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    x[i] = x[i + 1] = x[i + 2] = x[i + 3] = -INFINITY;
                    if (place(i) < read) sel_load4<BF>(from + i * stride, x + i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = place(i) < read ? sel_load<BF>(from + i * stride) : -INFINITY;
            }
        };
        if (a.bf16) load(std::true_type{}); else load(std::false_type{});
        float m = 0.f, inv = 1.f;
        if (row) {
            m = x[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
            m = sel_max<W>(m);
            if (m == -INFINITY) m = 0.f;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += sel_exp(x[i] - m);   // (a NaN stays one)
            inv = 1.f / sel_sum<W>(sum);
        }
        bool again = false;   // all of it in 64 bits
        uint32_t groups = ~0u;
        float top = 0.f;
        uint32_t key[V];
        if (scores) {
            // c, less the largest bias; -inf where there is no expert or none that may be picked
            float most_c = -INFINITY, least_x = INFINITY;
            bool odd = false;     // NaN or +inf
            auto sums = [&](auto sigmoid, auto biased) {
#pragma unroll
                for (int i = 0; i < V; i += VEC ? 4 : 1) {
                    float b[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (place(i) < held) {
                        if constexpr (!decltype(biased)::value) {
                            b[0] = b[1] = b[2] = b[3] = 0.f;
                        } else if constexpr (VEC) {
                            const float4 v = *reinterpret_cast<const float4*>(biases + e0 + place(i));
                            b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
                        } else {
                            b[0] = biases[e0 + place(i)];
                        }
#pragma unroll
                        for (int q = 0; q < (VEC ? 4 : 1); ++q) least_x = fminf(least_x, x[i + q]);
                    }
#pragma unroll
                    for (int q = 0; q < (VEC ? 4 : 1); ++q) {
                        float c = b[q];
                        if constexpr (decltype(sigmoid)::value) c += sel_sigmoid(x[i + q]);
                        else c += sel_exp(x[i + q] - m) * inv;
                        odd |= !(c < INFINITY);
                        most_c = fmaxf(most_c, c);
                        key[i + q] = __float_as_uint(c);
                    }
                }
            };
            if (a.sigmoid) {
                if (a.bias) sums(std::true_type{}, std::true_type{}); else sums(std::true_type{}, std::false_type{});
            } else {
                if (a.bias) sums(std::false_type{}, std::true_type{}); else sums(std::false_type{}, std::false_type{});
            }
            if (__any_sync(all, live && least_x == -INFINITY)) {   // excluded by their logits
                most_c = -INFINITY;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float c = __uint_as_float(key[i]);
                    if (place(i) < read && sel_value(a, t * a.E + e0 + place(i)) == -INFINITY) c = -INFINITY;
                    most_c = fmaxf(most_c, c);
                    key[i] = __float_as_uint(c);
                }
            }
            top = sel_max<W>(most_c);
            if (!(fabsf(top) < INFINITY)) top = 0.f;
            if (__any_sync(all, live && odd)) {   // keys cannot tell them
                again = live && odd;
#pragma unroll
                for (int o = W / 2; o; o >>= 1) again |= (bool)__shfl_xor_sync(all, (int)again, o);
            }
            bool stays = true;
            if (a.G > 1) {
                float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float c = __uint_as_float(key[i]);
                    m2 = fmaxf(m2, fminf(m1, c));
                    m1 = fmaxf(m1, c);
                }
                for (int o = 1; o < lpg; o <<= 1) {
                    const float o1 = __shfl_xor_sync(all, m1, o), o2 = __shfl_xor_sync(all, m2, o);
                    m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
                    m1 = fmaxf(m1, o1);
                }
                float value = m1;
                if (a.rank == 2) value += m2 != -INFINITY ? m2 : -top_bias;   // (sums of two, less the bias twice)
                const uint32_t vk = m1 == -INFINITY ? 0u : sel_key(value);
                int rank = 0;
                for (int g = 0; g < a.G; ++g) {
                    const uint32_t other = __shfl_sync(all, vk, (lane & ~(W - 1)) + (g << a.lpg_log2));
                    rank += other > vk || (other == vk && g < group);
                }
                stays = group < a.G && rank < a.kept && vk != 0u;
                // the least that stays and the largest that does not (0: only excluded ones)
                const uint32_t least = ~sel_max<W>(stays ? ~vk : 0u), most = sel_max<W>(stays || group >= a.G ? 0u : vk);
                const float lv = sel_unkey(least), mv = sel_unkey(most);
                // (each score is at most top + span, each c at most top, so that a sum's terms are at most it and 2 top)
                const float err = 4.f * sel_error(a.sigmoid, fabsf(top) + span) +
                                  2.f * kSelSum * (fabsf(lv) + fabsf(mv) + 4.f * fabsf(top) + (a.rank == 2 ? fabsf(top_bias) : 0.f));
                uint32_t border = __ballot_sync(all, live && most != 0u && !(lv - mv > err) && !again);
                while (border) {
                    const int owner = __ffs(border) - 1, base = owner & ~(W - 1);
                    border &= W == 32 ? 0u : ~(((1u << (W & 31)) - 1u) << base);
                    const float its = __shfl_sync(all, lv, owner), e2 = 2.f * __shfl_sync(all, err, owner);
                    const bool mine = (lane & ~(W - 1)) == base && group < a.G && vk != 0u;
                    const bool contends = mine && fabsf(value - its) <= e2;
                    const int sure = __popc(__ballot_sync(all, mine && lp == 0 && value > its + e2));
                    const float from = (a.rank == 2 && m2 != -INFINITY ? m2 : m1) - e2;
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float c = __uint_as_float(key[i]);
                        const bool in = contends && c >= from && c > -INFINITY;
                        const uint32_t votes = __ballot_sync(all, in);
                        const int at = n + __popc(votes & ((1u << lane) - 1u));
                        if (in && at < 32) rooms[warp].candidate[at] = e0 + place(i);
                        n += __popc(votes);
                    }
                    __syncwarp();
                    const float om = __shfl_sync(all, m, owner), oi = __shfl_sync(all, inv, owner);
                    const uint32_t mask = n <= 32 ? select_groups(a, first + part + owner / W, n, a.kept - sure, om, oi, &rooms[warp]) : 0u;
                    __syncwarp();
                    if ((lane & ~(W - 1)) == base && mask == 0u) again = true;
                    if (contends) stays = (mask >> group) & 1u;
                }
                groups = stays ? 1u << group : 0u;
#pragma unroll
                for (int o = W / 2; o; o >>= 1) groups |= __shfl_xor_sync(all, groups, o);
            }
            // keys by the distance from the largest: small ones are finer
            const float of = stays && live ? top : INFINITY;
            const uint32_t keep = ~low;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t d = __float_as_uint(of - __uint_as_float(key[i]));
                key[i] = (~d & keep) | ((code0 - (uint32_t)place(i)) & low);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = (sel_key(x[i]) & ~low) | ((code0 - (uint32_t)place(i)) & low);
        }
        // the picks and the one after them
        {
            constexpr int K = sel_kept<W, V>();
            uint32_t n[K];
#pragma unroll
            for (int j = 0; j < K; ++j) n[j] = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                uint32_t v = key[i];
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const uint32_t was = n[j];
                    n[j] = max(was, v);
                    v = min(was, v);
                }
            }
            if (gl == 0) tokens[warp][at_token] = {top, m, inv, again ? 0u : live ? groups : ~0u};
            uint32_t* mine = picks + at_token * (a.k + 1);
            for (int r = 0;; ++r) {
                const uint32_t best = sel_max<W>(n[0]);
                if (gl == 0) mine[r] = best;
                if (r == a.k) break;
                const bool won = n[0] == best;
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) n[j] = won ? n[j + 1] : n[j];
                n[K - 1] = won ? 0u : n[K - 1];
                if (__any_sync(all, n[0] == 0u)) {
                    uint32_t below = 0u - best;   // (that of 0, which is below every key)
#pragma unroll
                    for (int i = 0; i < V; ++i) below = max(below, key[i] - best);
                    if (n[0] == 0u && best) n[0] = best + below;
                }
            }
        }
    }
        __syncwarp();
        // A lane to a pick.  Neighbours that are too near each other first, then weights, relative to the largest of the
        // picks, so that small scores keep their digits.
        for (int q = 0; q < a.batch; q += per) {
            const int tk = q + lane / kp, j = lane & (kp - 1);
            const bool on = tk < a.batch && first + tk < a.T && j < a.k;
            const uint32_t* its = picks + tk * (a.k + 1) + j;
            uint32_t k0 = on ? its[0] : 0u, k1 = on ? its[1] : 0u;
            const SelToken token = tokens[warp][tk & 31];
            if (k0 < none) k0 = 0u;
            int e = k0 ? (int)(low - (k0 & low)) : -1;
            float xj = k0 ? sel_value(a, (first + tk) * a.E + e) : -INFINITY;
            bool near = false;
            if (scores) {
                // The sums of neighbours inside in full; the last pick's and the one behind it, of which there is the key.
                // (Equal logits and biases inside are in the order of their index.)
                const float bj = a.bias && k0 ? biases[e] : 0.f, sj = a.sigmoid ? sel_sigmoid(xj) : sel_exp(xj - token.max) * token.inv;
                const float d0 = token.top - (sj + bj), xn = __shfl_down_sync(all, xj, 1), bn = __shfl_down_sync(all, bj, 1);
                const float dn = __shfl_down_sync(all, d0, 1);
                const bool inside = j + 1 < a.k;
                const float d1 = inside ? dn : __uint_as_float(~k1 & ~low);
                near = k0 && k1 >= none && !(inside && xj == xn && bj == bn) &&
                       !(d1 - d0 > sel_margin(a, token.top, d1, a.sigmoid ? 1.f : sj + span, inside ? 0.f : a.quantum));
            } else if (!a.bf16) {
                near = k0 && k1 >= none && ((k0 ^ k1) & ~low) == 0u;
                // (equal ones inside too; at the end another, larger one may follow)
                const float xn = __shfl_down_sync(all, xj, 1);
                if (j + 1 < a.k && xj == xn) near = false;
            }
            const bool unknown = on && token.groups == 0u;
            if (__any_sync(all, near || unknown)) {
                const uint32_t votes = __ballot_sync(all, near), lost = __ballot_sync(all, unknown);
                for (int p = 0; p < per; ++p) {
                    const uint32_t segment = kp == 32 ? ~0u : (1u << kp) - 1u;
                    const uint32_t open = (votes >> (p * kp)) & segment, whole = (lost >> (p * kp)) & segment;
                    if (open || whole)
                        select_again(a, first + q + p, whole ? 0u : open, tokens[warp][q + p], span, top_bias, low, none, &rooms[warp],
                                     picks + (q + p) * (a.k + 1));
                }
                __syncwarp();
                k0 = on ? its[0] : 0u;
                if (k0 < none) k0 = 0u;
                e = k0 ? (int)(low - (k0 & low)) : -1;
                xj = k0 ? sel_value(a, (first + tk) * a.E + e) : -INFINITY;
            }
            float u = 0.f;
            if (a.renorm) {
                const float z = a.sigmoid ? fminf(xj, 0.f) : xj;
                const float base = sel_segment_max(z, kp);
                if (k0) u = sel_exp(z - base);
                if (k0 && row && isnan(token.inv)) u = NAN;   // a NaN beside the picks
                if (a.sigmoid && k0) u = xj == xj ? __fdividef(u, 1.f + sel_exp(-fabsf(xj))) : xj;   // (fminf drops a NaN)
                const float total = sel_segment_sum(u, kp);
                if (k0) u = __fdividef(u, total);
            } else if (k0) {
                u = a.sigmoid ? sel_sigmoid(xj) : sel_exp(xj - token.max) * token.inv;
            }
            if (on) {
                const long long at = (first + tk) * a.k + j;
                a.idx[at] = e;
                a.w[at] = u * a.scale;
            }
        }
        __syncwarp();
    }
}

// ---- backward --------------------------------------------------------------------------------------------------
// With D = sum_i w_i dw_i over the picks:
//   sigmoid                 dl_j = w_j (dw_j - D / scale) (1 - s_j), without the D where weights are not renormalised
//   softmax, renormalised   dl_j = w_j (dw_j - D / scale)
//   softmax, not            dl_e = -s_e D, and + w_j dw_j at the picks
// The first two touch the picks alone: a block keeps tiles of zeros in shared memory, puts a tile's picks in, sends it
// off as one bulk copy (tokens' rows follow one another) and takes the picks out again, so that a row costs k stores
// and no instruction for its zeros.
struct SelItem {
    int e;
    float d;
};
// pick j of token t (j over kp lanes of the token); D over the segment
__device__ __forceinline__ SelItem sel_grad(const SelectGradArgs& a, long long t, int j, bool on, int kp) {
    int e = -1;
    float w = 0.f, dw = 0.f, keep = 1.f;
    if (on) {
        e = __ldg(a.idx + t * a.k + j);
        if ((unsigned)e >= (unsigned)a.E) e = -1;
    }
    if (e >= 0) {
        w = __ldg(a.w + t * a.k + j);
        dw = __ldg(a.dw + t * a.k + j);
        if (a.sigmoid) {
            const float x = a.bf16 ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(a.logits) + t * a.E + e))
                                   : __ldg(static_cast<const float*>(a.logits) + t * a.E + e);
            keep = 1.f / (1.f + expf(x));
        }
    }
    const float D = a.renorm ? sel_segment_sum(w * dw, kp) * a.inv_scale : 0.f;
    return {e, w * (dw - D) * keep};
}

template <bool BF>
__global__ void __launch_bounds__(256) select_bwd_sparse_kernel(const SelectGradArgs a) {
    grid_dep_wait();
    extern __shared__ __align__(128) unsigned char sel_tiles[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int es = BF ? 2 : 4;
    const uint32_t tile_bytes = (uint32_t)a.tile * a.E * es;     // a multiple of 16
    for (uint32_t i = threadIdx.x * 16; i < 2 * tile_bytes; i += 256 * 16)
        *reinterpret_cast<uint4*>(sel_tiles + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int kp = 1;
    while (kp < a.k) kp *= 2;
    const int per = 32 / kp;
    int slot = 0, used = 0;
    for (long long tile = blockIdx.x; tile * a.tile < a.T; tile += gridDim.x, slot ^= 1, ++used) {
        const long long t0 = tile * a.tile;
        const int tokens = (int)min((long long)a.tile, a.T - t0);
        unsigned char* buf = sel_tiles + slot * tile_bytes;
        if (used >= 2) {   // the copy of two tiles ago has been read; its picks go
            if (threadIdx.x == 0) bulk_wait_read<1>();
            __syncthreads();
            const long long old = (tile - 2 * (long long)gridDim.x) * a.tile;
            for (int i = threadIdx.x; i < a.tile * a.k; i += 256) {
                const int e = __ldg(a.idx + old * a.k + i);
                if ((unsigned)e < (unsigned)a.E) {
                    const int at = i / a.k * a.E + e;
                    if constexpr (BF) reinterpret_cast<__nv_bfloat16*>(buf)[at] = __float2bfloat16(0.f);
                    else reinterpret_cast<float*>(buf)[at] = 0.f;
                }
            }
            __syncthreads();
        }
        for (int q = warp * per; q < tokens; q += 8 * per) {
            const int tk = q + lane / kp, j = lane & (kp - 1);
            const SelItem g = sel_grad(a, t0 + tk, j, tk < tokens && j < a.k, kp);
            if (g.e >= 0) {
                if constexpr (BF) reinterpret_cast<__nv_bfloat16*>(buf)[tk * a.E + g.e] = __float2bfloat16(g.d);
                else reinterpret_cast<float*>(buf)[tk * a.E + g.e] = g.d;
            }
        }
        fence_proxy_async_cta();
        __syncthreads();
        unsigned char* out = static_cast<unsigned char*>(a.dlogits) + t0 * a.E * es;
        const uint32_t bytes = (uint32_t)tokens * a.E * es, whole = bytes & ~15u;
        if (threadIdx.x == 0 && whole) {
            bulk_store(out, buf, whole);
            bulk_commit();
        }
        if (threadIdx.x * 2 < bytes - whole)   // the last tile's end
            reinterpret_cast<uint16_t*>(out + whole)[threadIdx.x] = reinterpret_cast<const uint16_t*>(buf + whole)[threadIdx.x];
    }
    if (threadIdx.x == 0) bulk_wait_all();
}

// dlogits += the gradient where only picks have one
__global__ void __launch_bounds__(256) select_bwd_add_kernel(const SelectGradArgs a) {
    grid_dep_wait();
    int kp = 1;
    while (kp < a.k) kp *= 2;
    const int lane = threadIdx.x & 31, per = 32 / kp;
    const long long t = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * per + lane / kp;
    const int j = lane & (kp - 1);
    const SelItem g = sel_grad(a, t, j, t < a.T && j < a.k, kp);
    if (g.e >= 0) static_cast<float*>(a.dlogits)[t * a.E + g.e] += g.d;
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
static unsigned sel_grid(long long tokens, int per_block, int blocks_sm, int num_sms) {
    return (unsigned)std::max<long long>(1, std::min((tokens + per_block - 1) / per_block, (long long)num_sms * blocks_sm));
}
static int pow2_at_least(int v) {
    int p = 1;
    while (p < v) p *= 2;
    return p;
}
static int log2_of(int p) {
    int l = 0;
    while ((1 << l) < p) ++l;
    return l;
}

template <int W, int V, bool VEC>
static cudaError_t select_c(cudaStream_t st, SelectArgs a, int num_sms) {
    constexpr int NT = 32 / W;
    // where a batch has many tokens a warp takes as many as fill its lanes with picks
    const int per = 32 / pow2_at_least(a.k);
    a.batch = a.few ? NT : std::max(NT, per);
    const size_t smem = ((size_t)kSelWarps * a.batch * (a.k + 1) + (a.bias ? (a.E + 3) / 4 * 4 : 0)) * 4;   // at most 21 KB
    const unsigned grid = sel_grid(a.T, kSelWarps * a.batch, V <= 16 ? 8 : V == 32 ? 4 : 2, num_sms);
    return launch_pdl(select_fwd_kernel<W, V, VEC>, grid, 32 * kSelWarps, smem, st, a);
}
template <int V, bool VEC>
static cudaError_t select_w(cudaStream_t st, const SelectArgs& a, int W, int num_sms) {
    if constexpr (V == 16) {
        switch (W) {
            case 1: return select_c<1, V, VEC>(st, a, num_sms);
            case 2: return select_c<2, V, VEC>(st, a, num_sms);
            case 4: return select_c<4, V, VEC>(st, a, num_sms);
            case 8: return select_c<8, V, VEC>(st, a, num_sms);
            case 16: return select_c<16, V, VEC>(st, a, num_sms);
        }
    }
    return select_c<32, V, VEC>(st, a, num_sms);
}
template <bool VEC>
static cudaError_t select_v(cudaStream_t st, const SelectArgs& a, int W, int V, int num_sms) {
    switch (V) {
        case 4: return select_w<4, VEC>(st, a, W, num_sms);
        case 8: return select_w<8, VEC>(st, a, W, num_sms);
        case 16: return select_w<16, VEC>(st, a, W, num_sms);
        case 32: return select_w<32, VEC>(st, a, W, num_sms);
    }
    return select_w<64, VEC>(st, a, W, num_sms);
}

cudaError_t launch_select_fwd(cudaStream_t st, SelectArgs a, int num_sms) {
    if (a.T == 0) return cudaSuccess;
    a.gs = a.E / a.G;
    const int bits = log2_of(a.E);
    a.low = (1u << bits) - 1u;
    a.quantum = (float)(1 << bits) * 1.1920929e-7f;   // what the last bits hold, relative to c
    // values a lane: 4 or 8 and a whole warp where there is less than a warp of tokens to fill an SM's schedulers with,
    // 16 otherwise; more where groups do not fit 32 lanes
    int V = 0, W = 32, lanes = 32;
    a.few = a.T <= 8 * num_sms;
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
    return a.gs % 4 == 0 ? select_v<true>(st, a, W, V, num_sms) : select_v<false>(st, a, W, V, num_sms);
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
    // tokens of a tile: a multiple of 8, so that a tile is one of 16 bytes; 8 KB or 8 tokens
    const int es = a.out_bf16 ? 2 : 4;
    a.tile = std::max(8, std::min(64, 8192 / (a.E * es) / 8 * 8));
    const size_t smem = 2 * (size_t)a.tile * a.E * es;   // at most 64 KB
    auto kern = a.out_bf16 ? select_bwd_sparse_kernel<true> : select_bwd_sparse_kernel<false>;
    static PerDevice<int> allowed[2];
    int dev = 0, done = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = allowed[a.out_bf16].get(dev, &done, [&](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, sel_grid(a.T, a.tile, smem > 32768 ? 3 : 6, num_sms), 256, smem, st, a);
}

cudaError_t launch_select_bias(cudaStream_t st, const int* counts, int B, int E, float* bias, float rate) {
    return launch_pdl(select_bias_kernel, 1, 1024, 0, st, counts, B, E, bias, rate);
}

}  // namespace moe
