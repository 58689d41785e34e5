// select_fwd.cuh - routing by scores, forward: each token's k experts by the scores of all of them, with a bias that only the
// choice sees and with groups of experts.  (Gradient, bias step and launches: select.cu.)
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
//
// What fp32 may be off by, and where each counts.  t is the largest finite bias, b - t a bias as it is kept, c a sum of it and a
// score, d = top - c its distance from the row's largest, u = 2^-24:
//
//   a score                  sel_error(its size), below                          each of two sums that are compared
//   b - t                    u |b - t| <= u (|c| + s); u s is within sel_error's   kSelSum |c| = 2 u |c|, with the next
//                            slack (sigmoid 3e-7 of at most 1.6e-7, softmax
//                            9e-7 s of 7.2e-7 s)
//   c                        u |c|, |c| <= |top| + d                              (above)
//   d                        u d                                                 kSelSum d
//   the index in d's bits    quantum d = 2^bits 2^-23 d, bits = log2 of E           where keys alone are compared
//   64 bits, b not less t    2 x 2^-53 |t| and what it takes from c               last = 1e-15 |t| (groups, two terms each: 4e-15 |t|)
//
//   two sums (sel_margin)         2 sel_error + 2 kSelSum (|top| + d) + (q + kSelSum) d + last, d the larger distance; q is
//       0 between picks, whose sums are made again in full; quantum where one is in full and one a key (the last pick and the
//       one behind it); 2 quantum for two keys (which neighbours hang together); 3 quantum where more picks are looked for,
//       so that none is missed that the finer tests then ask for.  An expert further than twice a margin behind the first
//       that was left out (select_again) cannot come before a pick.
//   scores of at most             1 (sigmoid), 1 / the row's sum (softmax), and of two neighbours s_j + span: s_(j+1) is at most
//       s_j + b_j - b_(j+1), span the finite biases' largest difference; of a group's terms |top| + span
//   two groups (sel_group_margin) 4 sel_error + 2 kSelSum (|v| + |w| + 4 |top| + |t| where one expert stands for two) + 4e-15 |t|;
//       a group's two terms and their sum v round by u (2 |m1| + 2 |m2| + |v|) <= u (3 |v| + 4 |top|) at most, as m1 <= top and
//       |m1| + |m2| = |v| or, of unlike signs, |m2| <= |v| + |top|
//   64 bits over a softmax's fp32 sum  2 sum_error |s - s'| (its error stands in both) + 1e-15 (|c| + |b|)
//   beyond fp32                   a bias that is -inf only less t, a group's sum that is -inf, a NaN, +inf: all in 64 bits (select_all)
//
// A change to a key's bits, to a sum's order or to sel_score64 changes these.
//
// Every call of the warp (__shfl_sync, __ballot_sync, __any_sync, the reductions) is made by all 32 lanes: none stands behind &&,
// || or ?: of a lane's own value, where lanes that have their answer would not take part, which is undefined.
//
// Bound by instruction issue: 131,072 x 512 (sigmoid, bias, k = 8) takes 110 us, 756 instructions a token at three quarters
// of the issue slots, where its logits take 42 us to read; 16,384 x 256 in 8 groups 18.7 us, of which about 5 are the tail
// that a token gone through again leaves (3 us each, most of it waiting for code and 64-bit arithmetic).
#pragma once
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

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
//   softmax: s (2^-22 + 2^-23 (-ln s)) and the sum's error, 2^-24 for each of V / 4 additions one after the other and some 2^-21
//            with the tree's and the exponentials'; s (-ln s) is at most 0.37
// Scores under 2^-126 = 1.18e-38 are 0 (the quotient's least number; a power over 2^128 is infinite), and among numbers under
// that a key's index takes 2^bits 2^-149 whatever their size: no score counts as smaller than 1.2e-33, 1.1e-5 of which is more.
__device__ __forceinline__ float sel_error(const SelectArgs& a, float most) {
    const float s = fminf(fmaxf(most, 1.2e-33f), 1.f);
    return a.sigmoid ? fminf(3e-7f, 1.1e-5f * s) : a.sum_error * s + fminf(4.5e-8f, 1.1e-5f * s);
}
constexpr float kSelSum = 1.2e-7f;   // of a sum's size: a rounding of it, and one of its bias less the largest

__device__ __forceinline__ float sel_max3(float a, float b, float c) {   // one instruction; passes over NaN as fmaxf does
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int W>
__device__ __forceinline__ float sel_max(float v) {
    if constexpr (W == 32) {
        float r;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    }
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

// The score of logit x in 64 bits, in the order and roundings of its formula; a softmax's with the row's largest logit and
// 1 / sum.  The code from here to the forward runs for a few tokens of a thousand and mostly waits for its own
// instructions and for 64-bit ones (a 64th of the rate), so it is kept short and out of line, its loops rolled.
static __device__ __noinline__ double sel_score64(bool sigmoid, float x, double row_max, double inv_sum) {
    const double z = exp(sigmoid ? -(double)x : (double)x - row_max);
    return sigmoid ? 1.0 / (1.0 + z) : z * inv_sum;
}

struct SelRoom {              // a warp's shared memory
    int candidate[32];
};
struct SelToken {             // what the forward found out about a token
    float top;                // its largest c, less the largest bias
    float last;               // what 64 bits may round from a sum with that bias back in
    float max, inv;           // of the softmax: the largest logit and 1 / sum
    uint32_t groups;          // bits of those that stay
    int doubt;                // 1: whether it is these; 2: of everything (a NaN, an infinity)
    int behind;               // picks after the last that were looked for too: 1, or 1 + kSelBehind where the first is near
};
constexpr int kSelBehind = 3;

struct SelOpen {              // one that is to be gone through again
    int t;
    uint32_t open;            // bit j: picks j and j + 1 are too near each other
    SelToken token;
};

// How far two sums may come nearer to each other than they are in fp32: scores of at most `most`, roundings of sums, biases
// and distances from `top`, of which d is the larger; `last` is what sums in 64 bits, which are what counts, lose; `quantum`
// is what the index has taken from d, if anything.
__device__ __forceinline__ float sel_margin(const SelectArgs& a, float top, float last, float d, float most, float quantum) {
    return 2.f * sel_error(a, most) + 2.f * kSelSum * (fabsf(top) + d) + (quantum + kSelSum) * d + last;
}

// The sum of a softmax's exponentials in 64 bits.
static __device__ __noinline__ double select_sum(const SelectArgs& a, long long t, double row_max) {
    double sum = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) sum += sel_score64(false, sel_value(a, t * a.E + e), row_max, 1.0);
#pragma unroll 1
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// Every expert in 64 bits, their groups too: k rounds of the largest that is left.
static __device__ __noinline__ void select_all(const SelectArgs& a, long long t, uint32_t low, uint32_t* picks) {
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
        sum = select_sum(a, t, top);
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
        if (scores) c = sel_score64(a.sigmoid, x, top, inv) + (double)b;
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
// that may be; their sums in 64 bits (without a bias their logits) decide.  A softmax's have its fp32 sum, whose error
// stands in both of two terms and so counts with their difference alone; where that is not enough, its sum is made in 64 bits
// (4097 x 999, k = 31: one such token of a batch made its forward 170 us instead of 79, by going through all experts).  Where
// there are more than 32, all experts are gone through.
static __device__ __noinline__ void select_again(const SelectArgs& a, long long t, uint32_t open, const SelToken& token, float top_bias,
                                                 uint32_t low, uint32_t none, SelRoom* room, uint32_t* picks) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const int from = __ffs(open) - 1;
    int n = min(33 - __clz(open), a.k) - from;
    if (lane < n) room->candidate[lane] = (int)(low - (picks[from + lane] & low));
    if ((open >> (a.k - 1)) & 1u) {
        const uint32_t next = picks[a.k];
        // (every score is at most 1; a softmax's at most 1 / its sum)
        const float d = __uint_as_float(~next & ~low);
        const float far = d + 2.f * sel_margin(a, token.top, token.last, d, a.sigmoid ? 1.f : token.inv, a.quantum);
        const uint32_t it = lane < token.behind ? picks[a.k + lane] : 0u;
        const bool may = it >= none && (a.bias ? __uint_as_float(~it & ~low) <= far : ((it ^ next) & ~low) == 0u);
        const int count = __popc(__ballot_sync(all, may));
        if (count < token.behind) {   // the last that was looked for is far enough, or there is none
            if (may && n + lane < 32) room->candidate[n + lane] = (int)(low - (it & low));
            n += count;
        } else {
        const int mine = lane < a.k ? (int)(low - (picks[lane] & low)) : -1;
#pragma unroll 4
        for (int i = 0; i < a.E; i += 32) {
            const int e = i + lane;
            bool in = false;
            if (e < a.E && (a.G == 1 || ((token.groups >> (e / a.gs)) & 1u))) {
                const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) - top_bias : 0.f;
                if (a.bias) in = x != -INFINITY && token.top - ((a.sigmoid ? sel_sigmoid(x) : sel_exp(x - token.max) * token.inv) + b) <= far;
                else in = (sel_key(x) & ~low) >= (next & ~low);
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
    }
    __syncwarp();
    if (n <= 32) {
        const int e = lane < n ? room->candidate[lane] : 0;
        const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) : 0.f;
        double inv = (double)token.inv;
#pragma unroll 1
        for (bool exact = !a.bias || a.sigmoid;; exact = true) {
            const double s = a.bias ? sel_score64(a.sigmoid, x, (double)token.max, inv) : 0.0, c = a.bias ? s + (double)b : (double)x;
            const uint64_t key = sel_key64(c);
            int rank = 0;
            bool near = false;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const uint64_t other = __shfl_sync(all, key, i);
                const int oe = __shfl_sync(all, e, i);
                rank += other > key || (other == key && oe < e);
                if (!exact) {
                    const double oc = __shfl_sync(all, c, i), os = __shfl_sync(all, s, i);
                    const float ox = __shfl_sync(all, x, i), ob = __shfl_sync(all, b, i);
                    near |= lane < n && i != lane && !(x == ox && b == ob) && !(fabs(c - oc) > 2.0 * a.sum_error * fabs(s - os) + 1e-15 * (fabs(c) + fabs(b)));
                }
            }
            if (exact || !__any_sync(all, near)) {
                if (lane < n && from + rank < a.k) picks[from + rank] = sel_pick(e, low);
                __syncwarp();
                return;
            }
            inv = 1.0 / select_sum(a, t, (double)token.max);
        }
    }
    select_all(a, t, low, picks);
}

// How far two groups' sums may come nearer to each other than they are in fp32: of two terms each, each at most 2 |top| and the
// sum in size, with a score of at most `most`.
// partial: a group of one expert has the largest bias taken off its sum once more, which rounds.
__device__ __forceinline__ float sel_group_margin(const SelectArgs& a, float top, float most, float top_bias, bool partial, float v, float w) {
    return 4.f * sel_error(a, most) +
           2.f * kSelSum * (fabsf(v) + fabsf(w) + 4.f * fabsf(top) + (partial ? fabsf(top_bias) : 0.f)) + 4e-15f * fabsf(top_bias);
}
// No softmax's score is above 1 / its sum, however far biases have spread.
__device__ __forceinline__ float sel_most(const SelectArgs& a, float most, float inv) { return a.sigmoid ? most : fminf(most, inv); }

// A token whose groups at the border are too near each other: which stay, from the sums in 64 bits of those alone that may.
// values: G sums as the forward has them (less the bias), then the least term of each (-inf: an excluded group).  0
// where that leaves it open (more than 32 experts may be terms; a softmax's sum has 32 bits; a sum is beyond 32 bits).
static __device__ __noinline__ uint32_t select_groups(const SelectArgs& a, long long t, const float* values, const SelToken& token, float span,
                                                      float top_bias, SelRoom* room) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const float value = lane < a.G ? values[lane] : 0.f, least_term = lane < a.G ? values[a.G + lane] : -INFINITY;
    const uint32_t vk = least_term == -INFINITY ? 0u : sel_key(value);
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.G; ++g) {
        const uint32_t other = __shfl_sync(all, vk, g);
        rank += other > vk || (other == vk && g < lane);
    }
    const bool stays = rank < a.kept && vk != 0u;
    const float lv = sel_unkey(~__reduce_max_sync(all, stays ? ~vk : 0u)), mv = sel_unkey(__reduce_max_sync(all, stays ? 0u : vk));
    const float e2 = 2.f * sel_group_margin(a, token.top, sel_most(a, fabsf(token.top) + span, token.inv), top_bias, a.rank == 2, lv, mv);
    // (two biases near the least number that there is add up to -inf, and no difference of those tells which is larger)
    if (!(e2 < INFINITY)) return 0u;
    const float over = value - lv;   // (one difference for both, so that none falls between them)
    const uint32_t sure = __ballot_sync(all, vk != 0u && over > e2), open = __ballot_sync(all, vk != 0u && !(over > e2) && over >= -e2);
    int n = 0;
#pragma unroll 1
    for (uint32_t rest = open; rest; rest &= rest - 1) {
        const int g = __ffs(rest) - 1;
        const float from = __shfl_sync(all, least_term, g) - e2;
#pragma unroll 1
        for (int i = lane; i < (a.gs + 31) / 32 * 32; i += 32) {
            const int e = g * a.gs + i;
            bool in = false;
            if (i < a.gs) {
                const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) - top_bias : 0.f;
                const float c = (a.sigmoid ? sel_sigmoid(x) : sel_exp(x - token.max) * token.inv) + b;
                in = x != -INFINITY && c >= from && c > -INFINITY;
            }
            const uint32_t votes = __ballot_sync(all, in);
            const int at = n + __popc(votes & ((1u << lane) - 1u));
            if (in && at < 32) room->candidate[at] = e;
            n += __popc(votes);
        }
    }
    if (n > 32) return 0u;
    __syncwarp();
    const int e = lane < n ? room->candidate[lane] : 0, g = lane < n ? e / a.gs : -1 - lane;
    const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) : 0.f;
    const double s = sel_score64(a.sigmoid, x, (double)token.max, (double)token.inv), c = s + (double)b;
    const uint64_t key = sel_key64(c);
    int place = 0;   // in its group
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint64_t other = __shfl_sync(all, key, i);
        const int oe = __shfl_sync(all, e, i), og = __shfl_sync(all, g, i);
        place += og == g && (other > key || (other == key && oe < e));
    }
    // the group's first candidate has its sum, with its second, if it has one
    const bool first = lane < n && place == 0;
    double sum = c, score = s;
    if (a.rank == 2) {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const double oc = __shfl_sync(all, c, i), os = __shfl_sync(all, s, i);
            const int og = __shfl_sync(all, g, i), op = __shfl_sync(all, place, i);
            if (first && og == g && op == 1) {
                sum = c + oc;
                score = s + os;
            }
        }
    }
    const int slots = a.kept - __popc(sure);
    int order = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const double os = __shfl_sync(all, sum, i);
        const int og = __shfl_sync(all, g, i);
        const bool of = __shfl_sync(all, (int)first, i);
        order += of && (os > sum || (os == sum && og < g));
    }
    if (!a.sigmoid) {
        bool near = false;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const double os = __shfl_sync(all, sum, i), oc = __shfl_sync(all, score, i);
            const bool in = __shfl_sync(all, (int)(first && order < slots), i);
            near |= first && order >= slots && in && !(os - sum > 2.0 * a.sum_error * fabs(oc - score) + 1e-15 * (fabs(os) + 1.0));
        }
        if (__any_sync(all, near)) return 0u;
    }
    return sure | __reduce_or_sync(all, first && order < slots ? 1u << g : 0u);
}

// Its picks when the groups turn out to be others: the k + 1 largest fp32 sums of `groups`, as the forward has them; returns
// how many there are.
static __device__ __noinline__ int select_picks(const SelectArgs& a, long long t, const SelToken& token, uint32_t groups, float top_bias, uint32_t low,
                                                uint32_t none, uint32_t* picks) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    uint32_t last = 0u;
    int count = 0;
#pragma unroll 1
    for (int r = 0; r <= a.k; ++r) {
        uint32_t best = 0u;
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) {
            if (!((groups >> (e / a.gs)) & 1u)) continue;
            const float x = sel_value(a, t * a.E + e), b = a.bias ? __ldg(a.bias + e) - top_bias : 0.f;
            uint32_t key;
            if (a.bias) {
                const float c = x == -INFINITY ? -INFINITY : (a.sigmoid ? sel_sigmoid(x) : sel_exp(x - token.max) * token.inv) + b;
                key = ~__float_as_uint(fmaxf(token.top - c, 0.f));
            } else {
                key = sel_key(x);
            }
            key = (key & ~low) | (low - (uint32_t)e);
            if (r == 0 || key < last) best = max(best, key);   // (expert 0 as the largest has every bit set)
        }
        last = __reduce_max_sync(all, best);
        if (lane == 0) picks[r] = last;
        count += last >= none;
        if (last == 0u) last = 1u;   // (nothing is below it)
    }
    __syncwarp();
    return count;
}

// ---- forward ---------------------------------------------------------------------------------------------------
// Keys that a lane keeps in order.  The k picks of a token fall on its W lanes; a lane that has given all it kept looks
// through its V keys again, which the whole warp waits for.  Of a token on a whole warp hardly a lane gives more than
// three of up to 12 picks (7 % of tokens at k = 8), so there the rounds do without looking, a maximum and a step down in the
// lane that held it, and are gone through again where that was wrong (131,072 x 512: 113 -> 110 us; with fewer lanes a
// token more would have to be kept, and 16,384 x 128 takes 8.1 us instead of 6.9).
constexpr int kSelOnce = 12, kSelOnceKept = 3;
template <int W, int V>
constexpr int sel_kept() { return W == 32 && V <= 16 ? 2 : W >= 16 ? 3 : 4; }

// KIND: rows taken a value at a time; four at a time; four at a time with every lane's places full (no tests of them)
enum : int { kSelOdd = 0, kSelVec = 1, kSelFull = 2 };

template <int W, int V, int KIND>
__global__ void __launch_bounds__(32 * kSelWarps, V <= 16 ? 8 : V == 32 ? 4 : 2) select_fwd_kernel(const __grid_constant__ SelectArgs a) {
    grid_dep_wait();
    constexpr bool VEC = KIND != kSelOdd, FULL = KIND == kSelFull;
    constexpr int NT = 32 / W;   // tokens of a warp
    extern __shared__ __align__(16) float sel_shared[];
    __shared__ SelRoom rooms[kSelWarps];
    __shared__ SelToken tokens[kSelWarps][32];
    __shared__ SelOpen opens[kSelWarps][32];
    __shared__ float ends[2 * kSelWarps];
    const unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane % W;
    const int lpg = 1 << a.lpg_log2, group = gl >> a.lpg_log2, lp = gl & (lpg - 1);
    const uint32_t low = a.low;
    const bool scores = a.bias || a.G > 1;                 // the scores are needed
    const bool row = !a.sigmoid && (scores || !a.renorm);  // the softmax's sum is needed
    const uint32_t none = a.bias ? 0x80800000u : 0x00800000u;   // keys below it are no expert's
    float* biases = sel_shared;                            // less the largest
    const int stride_k = a.k + 1 + kSelBehind;             // a token's picks and those behind them
    uint32_t* picks = reinterpret_cast<uint32_t*>(sel_shared + (a.bias ? (a.E + 3) / 4 * 4 : 0)) + warp * (a.batch + a.room) * stride_k;
    uint32_t* open_picks = picks + a.batch * stride_k;
    float* values = reinterpret_cast<float*>(picks + (kSelWarps - warp) * (a.batch + a.room) * stride_k) + warp * (a.batch + a.room) * 2 * a.G;
    float* open_values = values + a.batch * 2 * a.G;       // (not there without groups)
    int kp = 1;                                            // lanes of a token where lanes take one pick each
    while (kp < a.k) kp *= 2;
    const int per = 32 / kp;

    float span = 0.f, top_bias = 0.f;                      // of the finite biases
    bool odd_bias = false;                                 // one is NaN or +inf, or finite and, less the largest, -inf
    bool rounded = false;                                  // one is not what it was, so that unlike ones may be equal
    if (a.bias) {
        float hi = -INFINITY, lo = INFINITY;
        for (int e = threadIdx.x; e < a.E; e += 32 * kSelWarps) {
            const float b = __ldg(a.bias + e);
            biases[e] = b;
            odd_bias |= !(b < INFINITY);
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
        bool rounds = false;
        for (int e = threadIdx.x; e < a.E; e += 32 * kSelWarps) {
            const float b = biases[e];
            float d = b - top_bias;
            if (d == -INFINITY && b != -INFINITY) {   // which excludes nobody: sums that keys cannot tell
                d = NAN;
                odd_bias = true;
            }
            biases[e] = d;
            rounds |= d + top_bias != b;
        }
        odd_bias = __syncthreads_or(odd_bias);
        rounded = __syncthreads_or(rounds);
    }
    const float last = 1e-15f * fabsf(top_bias);
    auto place = [&](int i) { return VEC ? 4 * (lp + lpg * (i >> 2)) + (i & 3) : lp + lpg * i; };
    const int e0 = group * a.gs;
    const int held = group < a.G ? a.gs : 0;               // places below it hold experts
    const uint32_t code0 = low - (uint32_t)e0;
    // The weight of pick j of token t, over kp lanes of the token, relative to the largest of the picks, so that small scores
    // keep their digits.
    auto put = [&](long long t, int j, bool on, uint32_t pick, float xj, const SelToken& token) {
        float u = 0.f;
        if (a.renorm) {
            const float z = a.sigmoid ? fminf(xj, 0.f) : xj;
            const float base = sel_segment_max(z, kp);
            if (pick) u = sel_exp(z - base);
            if (pick && row && isnan(token.inv)) u = NAN;   // a NaN beside the picks
            if (a.sigmoid && pick) u = xj == xj ? __fdividef(u, 1.f + sel_exp(-fabsf(xj))) : xj;   // (fminf drops a NaN)
            const float total = sel_segment_sum(u, kp);
            if (pick) u = __fdividef(u, total);
        } else if (pick) {
            u = a.sigmoid ? sel_sigmoid(xj) : sel_exp(xj - token.max) * token.inv;
        }
        if (on) {
            const long long at = t * a.k + j;
            a.idx[at] = pick ? (int)(low - (pick & low)) : -1;
            a.w[at] = u * a.scale;
        }
    };
    // A warp takes `batch` tokens, NT at a time, and then all of their picks at once.  Tokens that are to be gone through
    // again wait until it is through with its others, or has `room` of them: calls amid the loop above would cost every
    // token its registers (16,384 x 256 in 8 groups 19.2 us, 13.1 without any).
    const long long step = (long long)gridDim.x * kSelWarps * a.batch;
    long long first = ((long long)blockIdx.x * kSelWarps + warp) * a.batch;
    while (first < a.T) {
    int waiting = 0;
    for (; first < a.T && waiting + a.batch <= a.room; first += step) {
    for (int part = 0; part < a.batch; part += NT) {
        const int at_token = part + lane / W;
        const long long t = first + at_token;
        const bool live = t < a.T && !(a.mask && !__ldg(a.mask + t));
        const int read = live ? held : 0;
        float x[V];
        auto load = [&](auto bf) {   // (a copy of the loop for each type, so that none is chosen for each value)
            constexpr bool BF = decltype(bf)::value;
            const long long at = FULL ? min(t, (long long)a.T - 1) : t;   // (a full lane reads, whether it counts or not)
            const char* from = static_cast<const char*>(a.logits) + (at * a.E + e0 + place(0)) * (BF ? 2 : 4);
            const int stride = lpg * (BF ? 2 : 4);         // bytes between a lane's places (four times it if VEC)
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    if constexpr (!FULL) x[i] = x[i + 1] = x[i + 2] = x[i + 3] = -INFINITY;
                    if (FULL || place(i) < read) sel_load4<BF>(from + i * stride, x + i);
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
            for (int i = 1; i + 1 < V; i += 2) m = sel_max3(m, x[i], x[i + 1]);
            m = sel_max<W>(fmaxf(m, x[V - 1]));
            if (m == -INFINITY) m = 0.f;
            float part[4] = {0.f, 0.f, 0.f, 0.f};   // (four shorter sums round less than one)
#pragma unroll
            for (int i = 0; i < V; ++i) part[i & 3] += sel_exp(x[i] - m);   // (a NaN stays one)
            inv = 1.f / sel_sum<W>((part[0] + part[1]) + (part[2] + part[3]));
        }
        bool again = false, doubt = false;   // of everything, of the groups
        uint32_t groups = ~0u;
        float top = 0.f;
        uint32_t key[V];
        if (scores) {
            // c, less the largest bias; -inf where there is no expert or none that may be picked
            float most_c = -INFINITY;
            bool special = false;   // a logit that is NaN or infinite
            auto sums = [&](auto sigmoid, auto biased) {
#pragma unroll
                for (int i = 0; i < V; i += VEC ? 4 : 1) {
                    float b[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    if (FULL || place(i) < held) {
                        if constexpr (!decltype(biased)::value) {
                            b[0] = b[1] = b[2] = b[3] = 0.f;
                        } else if constexpr (VEC) {
                            const float4 v = *reinterpret_cast<const float4*>(biases + e0 + place(i));
                            b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
                        } else {
                            b[0] = biases[e0 + place(i)];
                        }
#pragma unroll
                        for (int q = 0; q < (VEC ? 4 : 1); ++q) special |= !(fabsf(x[i + q]) < INFINITY);
                    }
#pragma unroll
                    for (int q = 0; q < (VEC ? 4 : 1); ++q) {
                        float c = b[q];
                        if constexpr (decltype(sigmoid)::value) c += sel_sigmoid(x[i + q]);
                        else c += sel_exp(x[i + q] - m) * inv;
                        key[i + q] = __float_as_uint(c);
                    }
                    if constexpr (VEC) {
                        most_c = sel_max3(most_c, __uint_as_float(key[i]), __uint_as_float(key[i + 1]));
                        most_c = sel_max3(most_c, __uint_as_float(key[i + 2]), __uint_as_float(key[i + 3]));
                    } else {
                        most_c = fmaxf(most_c, __uint_as_float(key[i]));
                    }
                }
            };
            if (a.sigmoid) {
                if (a.bias) sums(std::true_type{}, std::true_type{}); else sums(std::true_type{}, std::false_type{});
            } else {
                if (a.bias) sums(std::false_type{}, std::true_type{}); else sums(std::false_type{}, std::false_type{});
            }
            if (odd_bias || __any_sync(all, live && special)) {
                // experts that are excluded by their logits; sums that are NaN or +inf, which keys cannot tell
                bool odd = false;
                most_c = -INFINITY;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float c = __uint_as_float(key[i]);
                    if (place(i) < read && sel_value(a, t * a.E + e0 + place(i)) == -INFINITY) c = -INFINITY;
                    odd |= !(c < INFINITY);
                    most_c = fmaxf(most_c, c);
                    key[i] = __float_as_uint(c);
                }
                again = live && odd;
#pragma unroll
                for (int o = W / 2; o; o >>= 1) again |= (bool)__shfl_xor_sync(all, (int)again, o);
            }
            top = sel_max<W>(most_c);
            if (!(fabsf(top) < INFINITY)) top = 0.f;
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
                const bool partial = a.rank == 2 && __any_sync(all, m1 != -INFINITY && m2 == -INFINITY);
                const float err = sel_group_margin(a, top, sel_most(a, fabsf(top) + span, inv), top_bias, partial, lv, mv);
                doubt = live && most != 0u && !(lv - mv > err);
                if (__any_sync(all, doubt) && lp == 0 && group < a.G) {   // (for select_groups)
                    values[at_token * 2 * a.G + group] = value;
                    values[(at_token * 2 + 1) * a.G + group] = vk == 0u ? -INFINITY : a.rank == 2 && m2 != -INFINITY ? m2 : m1;
                }
                groups = stays ? 1u << group : 0u;
#pragma unroll
                for (int o = W / 2; o; o >>= 1) groups |= __shfl_xor_sync(all, groups, o);
            }
            if (a.bias) {
                // keys by the distance from the largest: small ones are finer
                const float of = stays && live ? top : INFINITY;
                const uint32_t keep = ~low;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t d = __float_as_uint(of - __uint_as_float(key[i]));
                    const uint32_t code = code0 - (uint32_t)place(i);
                    key[i] = FULL ? (~d & keep) | code : (~d & keep) | (code & low);
                }
            } else {
                if (a.bf16) load(std::true_type{}); else load(std::false_type{});   // (the scores took their place)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    key[i] = stays && live && (FULL || place(i) < read) ? (sel_key(x[i]) & ~low) | ((code0 - (uint32_t)place(i)) & low) : 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = !FULL || live ? (sel_key(x[i]) & ~low) | ((code0 - (uint32_t)place(i)) & low) : 0u;
        }
        // the picks and the one after them
        {
            uint32_t* mine = picks + at_token * stride_k;
            int end = a.k;
            auto rounds = [&](auto kept, auto look) {
                constexpr int K = decltype(kept)::value;
                constexpr bool LOOK = decltype(look)::value;
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
                        if (j + 1 < K) v = min(was, v);
                    }
                }
                const bool more = n[K - 1] != 0u;   // than it keeps, perhaps
                uint32_t before = 0u;
                end = a.k;
#pragma unroll 4
                for (int r = 0;; ++r) {
                    const uint32_t best = sel_max<W>(n[0]);
                    if (gl == 0) mine[r] = best;
                    if (r == end) {
                        // where the first that is left is too near the last pick, a few more, so that it is known which
                        // may change places with it
                        if (end != a.k) break;
                        bool edge = best >= none;
                        if (a.bias) {
                            const float d = __uint_as_float(~best & ~low);
                            edge = edge && !(d - __uint_as_float(~before & ~low) > sel_margin(a, top, last, d, a.sigmoid ? 1.f : inv, 3.f * a.quantum));
                        } else {
                            edge = edge && ((best ^ before) & ~low) == 0u;
                        }
                        if (!__any_sync(all, edge && (a.bias || !a.bf16))) break;
                        end = a.k + kSelBehind;
                    }
                    before = best;
                    const bool won = n[0] == best;
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) n[j] = won ? n[j + 1] : n[j];
                    n[K - 1] = won ? 0u : n[K - 1];
                    if constexpr (LOOK) {
                        if (__any_sync(all, n[0] == 0u)) {
                            uint32_t below = 0u - best;   // (that of 0, which is below every key)
#pragma unroll
                            for (int i = 0; i < V; ++i) below = max(below, key[i] - best);
                            if (n[0] == 0u && best) n[0] = best + below;
                        }
                    }
                }
                return !LOOK && __any_sync(all, more && n[0] == 0u);
            };
            bool again_looking = true;
            if constexpr (W == 32 && V >= 16)   // (where tokens are few the code's own way to the SM counts)
                again_looking = a.k > kSelOnce || rounds(std::integral_constant<int, kSelOnceKept>{}, std::false_type{});
            if (again_looking) rounds(std::integral_constant<int, sel_kept<W, V>()>{}, std::true_type{});
            if (gl == 0) tokens[warp][at_token] = {top, last, m, inv, groups, again ? 2 : doubt ? 1 : 0, 1 + end - a.k};
        }
    }
        __syncwarp();
        // A lane to a pick: neighbours that are too near each other, weights.
        for (int q = 0; q < a.batch; q += per) {
            const int tk = q + lane / kp, j = lane & (kp - 1);
            const bool on = tk < a.batch && first + tk < a.T && j < a.k;
            const uint32_t* its = picks + tk * stride_k + j;
            uint32_t k0 = on ? its[0] : 0u;
            const uint32_t k1 = on ? its[1] : 0u;
            const SelToken token = tokens[warp][tk & 31];
            if (k0 < none) k0 = 0u;
            const int e = (int)(low - (k0 & low));
            const float xj = k0 ? sel_value(a, (first + tk) * a.E + e) : -INFINITY;
            bool near = false, equal = false, chain = false;
            if (a.bias) {
                // The sums of neighbours inside in full; the last pick's and the one behind it, of which there is the key.
                // (Equal logits and biases inside are in the order of their index.)
                const float bj = a.bias && k0 ? biases[e] : 0.f, sj = a.sigmoid ? sel_sigmoid(xj) : sel_exp(xj - token.max) * token.inv;
                const float d0 = token.top - (sj + bj), xn = __shfl_down_sync(all, xj, 1), bn = __shfl_down_sync(all, bj, 1);
                const float dn = __shfl_down_sync(all, d0, 1);
                const bool inside = j + 1 < a.k, both = k0 && k1 >= none;
                const float t0 = __uint_as_float(~k0 & ~low), t1 = __uint_as_float(~k1 & ~low), d1 = inside ? dn : t1;
                const float most = sel_most(a, a.sigmoid ? 1.f : sj + span, token.inv);
                near = both && !(d1 - d0 > sel_margin(a, token.top, last, d1, most, inside ? 0.f : a.quantum));
                equal = inside && xj == xn && bj == bn && !rounded;
                // (what is out of order may belong behind others whose keys are as near)
                chain = both && !(t1 - t0 > sel_margin(a, token.top, last, t1, most, 2.f * a.quantum));
            } else if (!a.bf16) {
                near = chain = k0 && k1 >= none && ((k0 ^ k1) & ~low) == 0u;
                // (equal ones inside too; at the end another, larger one may follow)
                const float xn = __shfl_down_sync(all, xj, 1);
                equal = j + 1 < a.k && xj == xn;
            }
            const bool unknown = on && token.doubt != 0;
            bool waits = false;
            if (__any_sync(all, (near && !equal) || unknown)) {
                const uint32_t unequal = __ballot_sync(all, near && !equal), votes = __ballot_sync(all, near || chain), lost = __ballot_sync(all, unknown);
                for (int p = 0; p < per; ++p) {
                    const uint32_t segment = kp == 32 ? ~0u : (1u << kp) - 1u;
                    // (equal neighbours alone are in order, but what follows them may belong before both)
                    const uint32_t open = (unequal >> (p * kp)) & segment ? (votes >> (p * kp)) & segment : 0u, whole = (lost >> (p * kp)) & segment;
                    if (!(open || whole)) continue;
                    if (lane / kp == p) waits = true;
                    if (lane == 0) opens[warp][waiting] = {(int)(first + q + p), open, tokens[warp][q + p]};
                    if (tokens[warp][q + p].doubt == 1)
                        for (int r = lane; r < 2 * a.G; r += 32) open_values[waiting * 2 * a.G + r] = values[(q + p) * 2 * a.G + r];
                    for (int r = lane; r < stride_k; r += 32) open_picks[waiting * stride_k + r] = picks[(q + p) * stride_k + r];
                    ++waiting;
                }
            }
            put(first + tk, j, on && !waits, k0, xj, token);
        }
        __syncwarp();
    }
    for (int i = 0; i < waiting; ++i) {
        SelOpen open = opens[warp][i];
        uint32_t* its = open_picks + i * stride_k;
        bool lost = open.token.doubt == 2;
        if (open.token.doubt == 1) {
            const uint32_t groups = select_groups(a, open.t, open_values + i * 2 * a.G, open.token, span, top_bias, &rooms[warp]);
            lost = groups == 0u;
            if (!lost && groups != open.token.groups) {
                open.token.groups = groups;
                open.token.behind = 1;
                const int pairs = min(a.k, select_picks(a, open.t, open.token, groups, top_bias, low, none, its) - 1);
                open.open = pairs <= 0 ? 0u : pairs >= 32 ? ~0u : (1u << pairs) - 1u;
            }
        }
        if (lost) select_all(a, open.t, low, its);
        else if (open.open) select_again(a, open.t, open.open, open.token, top_bias, low, none, &rooms[warp], its);
        const int j = lane & (kp - 1);
        uint32_t pick = j < a.k ? its[j] : 0u;
        if (pick < none) pick = 0u;
        const float xj = pick ? sel_value(a, (long long)open.t * a.E + (int)(low - (pick & low))) : -INFINITY;
        put(open.t, j, lane < a.k, pick, xj, open.token);
        __syncwarp();
    }
    }
}


// ---- launches --------------------------------------------------------------------------------------------------
inline unsigned sel_grid(long long tokens, int per_block, int blocks_sm, int num_sms) {
    return (unsigned)std::max<long long>(1, std::min((tokens + per_block - 1) / per_block, (long long)num_sms * blocks_sm));
}
inline int pow2_at_least(int v) {
    int p = 1;
    while (p < v) p *= 2;
    return p;
}
inline int log2_of(int p) {
    int l = 0;
    while ((1 << l) < p) ++l;
    return l;
}

template <int W, int V, int KIND>
static cudaError_t select_c(cudaStream_t st, SelectArgs a, int num_sms) {
    constexpr int NT = 32 / W;
    // Where there are many tokens a warp takes as many as fill its lanes with picks; not where that leaves an SM fewer than 16
    // warps (k = 8, four tokens against one or two: 4800 x 512 15.2 and 12.2 us, 9600 x 512 the same, 16,384 x 512 20.1 and 23.9).
    const int per = 32 / pow2_at_least(a.k);
    a.batch = a.few ? NT : std::max(NT, per);
    while (a.batch > NT && (a.batch * a.G > 256 || a.T < (long long)a.batch * 16 * num_sms)) a.batch /= 2;
    a.room = std::max(8, a.batch);
    a.sum_error = 9e-7f + 1.5e-8f * V;
    const size_t words = (size_t)kSelWarps * (a.batch + a.room) * (a.k + 1 + kSelBehind + (a.G > 1 ? 2 * a.G : 0));
    const size_t smem = (words + (a.bias ? (a.E + 3) / 4 * 4 : 0)) * 4;   // at most 33 KB
    const unsigned grid = sel_grid(a.T, kSelWarps * a.batch, V <= 16 ? 8 : V == 32 ? 4 : 2, num_sms);
    return launch_pdl(select_fwd_kernel<W, V, KIND>, grid, 32 * kSelWarps, smem, st, a);
}
template <int V, int KIND>
static cudaError_t select_w(cudaStream_t st, const SelectArgs& a, int W, int num_sms) {
    if constexpr (V == 16) {
        switch (W) {
            case 1: return select_c<1, V, KIND>(st, a, num_sms);
            case 2: return select_c<2, V, KIND>(st, a, num_sms);
            case 4: return select_c<4, V, KIND>(st, a, num_sms);
            case 8: return select_c<8, V, KIND>(st, a, num_sms);
            case 16: return select_c<16, V, KIND>(st, a, num_sms);
        }
    }
    return select_c<32, V, KIND>(st, a, num_sms);
}
// (each kind is a translation unit of its own: they take long to compile)
template <int KIND>
cudaError_t select_kind(cudaStream_t st, const SelectArgs& a, int W, int V, int num_sms) {
    switch (V) {
        case 4: return select_w<4, KIND>(st, a, W, num_sms);
        case 8: return select_w<8, KIND>(st, a, W, num_sms);
        case 16: return select_w<16, KIND>(st, a, W, num_sms);
        case 32: return select_w<32, KIND>(st, a, W, num_sms);
    }
    return select_w<64, KIND>(st, a, W, num_sms);
}

}  // namespace moe
