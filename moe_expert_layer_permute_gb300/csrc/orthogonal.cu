// orthogonal.cu - Newton-Schulz orthogonalisation of a batch of matrices: the update of the Muon
// optimiser for expert weights.
//
// For each matrix G [R, C]:  X = G / (|G|_F + eps), then `steps` times, with coefficients (a, b, c),
//   A = X X^T,   B = b A + c A A,   X <- a X + B X,
// on the side with the shorter edge: with m = min(R, C), n = max(R, C), X is kept as [m, n] (G^T where
// R > C) and A and B are m x m.
//
// Operands are fp16 and sums fp32.  Eleven significant bits at the full rate of the 16-bit MMA; bf16's
// eight left the result 1.5-7 % off the exact one (relative 2-norm).  fp16's range is covered by
// powers of two: X is held times 2^8, A and B times 2^10, and the first X is G times a power of two,
// exact for bf16 G; the rest of the norm, 1/s with s in [1/2, 1), enters the first step's epilogues in
// fp32.  Small singular values grow about 3.4-fold a step while X's rounding stays relative to its
// largest ones, so X also keeps its rounding error as a second fp16 (`lo`, times 2^11 again) for the
// a X term of every step but the last: without it gradients of low rank came out 1 % off, with it
// 0.1 %.  What A's and B's roundings do depends on G: the error of a singular value is their errors' mean over
// the entries that its vectors weigh, next to nothing where those are many, and the steps amplify it (the
// slope of the polynomial reaches 1.8).  A matrix of up to 128 rows keeps the rounding errors of A and B, as second
// products of POLY (A by twice its error, which along a singular vector is what both orders give) and of APPLY: 4 of
// 128 rows of 1024 values alone came out up to 6.8e-3 off without, 1.2e-3 with them (before the rounding to bf16),
// dense ones 1.5e-3 and 0.9e-3.  More rows would take 1.7 times the arithmetic (768 x 2048) and go without: 4 of
// 300 rows come out up to 6.3e-3 off, and a few entries, in any size, up to 1e-2, since X's own rounding in
// GRAM counts there.  In the large kernel the rest of a X goes through the
// products, as a on B's diagonal: the epilogue then needs no X (256 x 768 x 2048: 1 % less time), and the
// error moves between kinds of matrices (before the rounding to bf16, 200 x 600: gaussian 1.80 -> 1.56e-3,
// rank 25 0.8 -> 1.7e-3).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "per_device.h"
#include "slab.h"

#include <cuda_fp16.h>

namespace moe {

constexpr float kXScale = 256.f, kABScale = 1024.f, kLoScale = 2048.f;
constexpr int kNsStages = 4;
constexpr int kNsEpi = 8;          // epilogue warps: two for each quarter of the TMEM lanes, on alternate columns
constexpr int kNsThreads = 32 * (5 + kNsEpi);   // operand loads, MMA, the epilogue, watcher, box loads, box stores
constexpr int kNsSlots = 3;        // pairs of boxes between the box loads, the epilogue and the box stores
constexpr int kNsBox = 16384;      // a box: 128 rows x 64 16-bit values, 128-byte swizzle
constexpr int kNsSmem = 1024 + kNsStages * 32768 + kNsSlots * 2 * kNsBox + 512;
constexpr int kNormPart = 8192;    // elements of one partial sum of squares
constexpr int kNormParts = 512;    // most partial sums of a matrix

// ---- norms and the first X ---------------------------------------------------------------------------
__device__ __forceinline__ float ns_val(const float* p, long long i) { return __ldg(p + i); }
__device__ __forceinline__ float ns_val(const __nv_bfloat16* p, long long i) { return __bfloat162float(p[i]); }

__device__ __forceinline__ float ns_block_sum(float v) {   // 256 threads; the sum on every thread
    __shared__ float part[8];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[threadIdx.x & 7];
#pragma unroll
    for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    return v;
}

// eight consecutive values from a 16-byte boundary
__device__ __forceinline__ void ns_val8(float* v, const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ns_val8(float* v, const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_bf16x2(w[j]);
        v[2 * j] = f.x; v[2 * j + 1] = f.y;
    }
}

// Part blockIdx.x of matrix blockIdx.y's sum of squares: runs of eight from the first 16-byte boundary on, and
// by part 0 the few elements before and after them.
template <typename T>
__global__ void __launch_bounds__(256) ns_norm_kernel(const T* G, long long elems, int parts, float* partial) {
    grid_dep_wait();
    const T* g = G + (long long)blockIdx.y * elems;
    const long long head = min(elems, (long long)((16 - reinterpret_cast<uintptr_t>(g) % 16) % 16 / sizeof(T)));
    const long long runs = (elems - head) / 8;
    float v = 0.f;
#pragma unroll 4
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < runs; i += (long long)parts * 256) {
        float x[8];
        ns_val8(x, g + head + 8 * i);
        float s = x[0] * x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) s += x[j] * x[j];
        v += s;
    }
    if (blockIdx.x == 0) {
        const long long tail = head + 8 * runs;
        float x = 0.f;
        if (threadIdx.x < head) x = ns_val(g, threadIdx.x);
        else if (threadIdx.x >= 32 && tail + threadIdx.x - 32 < elems) x = ns_val(g, tail + threadIdx.x - 32);
        v += x * x;
    }
    v = ns_block_sum(v);
    if (threadIdx.x == 0) partial[(long long)blockIdx.y * parts + blockIdx.x] = v;
}

// The power of two p with |G| p in [1/2, 1) (1 for |G| = 0), and inv_s = 1 / ((|G| + eps) p), so that the
// first X is G p inv_s.  A norm that is not finite makes the whole matrix NaN.
__device__ __forceinline__ float ns_split(float norm, float eps, float* inv_s) {
    const int ex = (int)((__float_as_uint(norm) >> 23) & 0xffu) - 126;   // -62 .. 64: a root of an fp32 sum
    const bool fine = norm <= 3.4e38f;
    const bool none = norm < 1e-30f;
    const float p = none ? 1.f : __uint_as_float((uint32_t)(127 - ex) << 23);
    *inv_s = none ? 1.f : fine ? 1.f / ((norm + eps) * p) : NAN;   // (X is 0 then)
    return fine ? p : NAN;
}

struct NsPrep {
    const float* partial;
    __half* hi;
    __half* lo;      // null where G is exact in fp16 (bf16 G)
    float* inv_s;    // [N]
    int* done;       // [N][counts], zeroed
    int counts, parts, R, C, ld;
    float eps;
    int flip;        // store G^T
};

// The factor of matrix `mat`'s first X from its partial sums; `first` also records inv_s.
__device__ __forceinline__ float ns_factor(const NsPrep& a, int mat, bool first) {
    float v = 0.f;
    for (int i = threadIdx.x; i < a.parts; i += 256) v += a.partial[(long long)mat * a.parts + i];
    float inv_s;
    const float f = ns_split(sqrtf(ns_block_sum(v)), a.eps, &inv_s) * kXScale;
    if (first) {
        if (threadIdx.x == 0) a.inv_s[mat] = inv_s;
        for (int i = threadIdx.x; i < a.counts; i += 256) a.done[(long long)mat * a.counts + i] = 0;
    }
    return f;
}
__device__ __forceinline__ uint32_t ns_pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 ns_unpack_half(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
// a pair of values of X, and of their rounding errors
__device__ __forceinline__ uint32_t ns_split_pair(float x, float y, uint32_t* lo) {
    const uint32_t h = ns_pack_half(x, y);
    const float2 f = ns_unpack_half(h);
    *lo = ns_pack_half((x - f.x) * kLoScale, (y - f.y) * kLoScale);
    return h;
}
// a pair of values of A, and twice their rounding errors (see ns_small_kernel)
__device__ __forceinline__ uint32_t ns_split_a(float x, float y, uint32_t* twice) {
    const uint32_t h = ns_pack_half(x, y);
    float v[2] = {2.f * x, 2.f * y};
    fma_f16x2(v, h, 0xc000u);   // -2
    *twice = ns_pack_half(v[0], v[1]);
    return h;
}
// eight values of X, and their rounding errors, at a 16-byte boundary
__device__ __forceinline__ void ns_store8(const NsPrep& a, long long at, const float* x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = ns_split_pair(x[2 * j], x[2 * j + 1], l + j);
    *reinterpret_cast<uint4*>(a.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    if (a.lo) *reinterpret_cast<uint4*>(a.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

// The three kernels below request their part of G before they wait for the norms' kernel: it wrote none of
// G, and waited itself for what did.

// Rows of multiples of 8 elements, as they stand: X's pitch is C and the matrix one run of elements.
constexpr int kPrepPer = 4;   // runs of eight per thread
template <typename T>
__global__ void __launch_bounds__(256) ns_prep_kernel(const T* G, const NsPrep a) {
    const int mat = blockIdx.y;
    const long long elems = (long long)a.R * a.C;
    const long long i0 = ((long long)blockIdx.x * kPrepPer * 256 + threadIdx.x) * 8;
    float x[kPrepPer][8];
#pragma unroll
    for (int q = 0; q < kPrepPer; ++q)
        if (i0 + q * 2048 < elems) ns_val8(x[q], G + mat * elems + i0 + q * 2048);
    grid_dep_wait();
    const float f = ns_factor(a, mat, blockIdx.x == 0);
#pragma unroll
    for (int q = 0; q < kPrepPer; ++q) {
        if (i0 + q * 2048 >= elems) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[q][j] *= f;
        ns_store8(a, mat * elems + i0 + q * 2048, x[q]);
    }
}

// Other rows as they stand: runs of eight of X's rows, whose pitch is a multiple of eight; a row's last run
// is filled up with zeros.
template <typename T>
__global__ void __launch_bounds__(256) ns_prep_rows_kernel(const T* G, const NsPrep a) {
    const int mat = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x;   // R ld / 8 < 2^31
    const int row = i / (a.ld / 8), c = (i - row * (a.ld / 8)) * 8;
    const T* g = G + ((long long)mat * a.R + row) * a.C + c;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = row < a.R && c + j < a.C ? ns_val(g, j) : 0.f;
    grid_dep_wait();
    const float f = ns_factor(a, mat, blockIdx.x == 0);
    if (row >= a.R) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= f;
    ns_store8(a, ((long long)mat * a.R + row) * a.ld + c, x);
}

// G^T by tiles of 64 x 64 through shared memory, which holds fp16 pairs of two rows of G in the order that
// keeps both its writes and its reads free of bank conflicts (32 x 2048 x 768, bf16: 40 us, 5 TB/s; with single
// fp32 values there 46).  VEC: rows of multiples of 8 elements, loaded 16 bytes at a time.  Stores are 32
// bytes (the pitch is a multiple of 16 bytes; what is past R in a row's last 16 is never read).  A block goes
// down `per` tiles, the next one's loads under way while one is stored.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) ns_prep_flip_kernel(const T* G, const NsPrep a, int per) {
    constexpr bool kLo = sizeof(T) == 4;
    __shared__ uint32_t tile[kLo ? 2 : 1][32][65];
    const int mat = blockIdx.z, c0 = blockIdx.x * 64;
    // loads: VEC: rows 2 lp, 2 lp + 1, columns lc ..; else rows 2 (lp + 8 q) .., columns lc, lc + 32
    const int lp = threadIdx.x >> (VEC ? 3 : 5), lc = VEC ? (threadIdx.x & 7) * 8 : threadIdx.x & 31;
    const int c = threadIdx.x >> 2, rp = (threadIdx.x & 3) * 8;    // stores: row pairs rp .. of column c
    float x[2][8];
    auto load = [&](int r0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (VEC) {
                const int r = r0 + 2 * lp + h;
                if (r < a.R && c0 + lc < a.C) {
                    ns_val8(x[h], G + ((long long)mat * a.R + r) * a.C + c0 + lc);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[h][j] = 0.f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = r0 + 2 * (lp + 8 * (j >> 1)) + h, col = c0 + lc + 32 * (j & 1);
                    x[h][j] = r < a.R && col < a.C ? ns_val(G, ((long long)mat * a.R + r) * a.C + col) : 0.f;
                }
            }
        }
    };
    const int first = blockIdx.y * 64 * per, end = min(a.R, first + 64 * per);
    load(first);
    grid_dep_wait();
    const float f = ns_factor(a, mat, blockIdx.x == 0 && blockIdx.y == 0);
    for (int r0 = first; r0 < end; r0 += 64) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t lo;
            if constexpr (VEC) {   // columns 32 apart are in one bank: one half goes the other way round
                const bool far = lc >= 32;
                const int col = lc + (far ? j ^ 4 : j);
                tile[0][lp][col] = ns_split_pair((far ? x[0][j ^ 4] : x[0][j]) * f, (far ? x[1][j ^ 4] : x[1][j]) * f, &lo);
                if constexpr (kLo) tile[1][lp][col] = lo;
            } else {
                tile[0][lp + 8 * (j >> 1)][lc + 32 * (j & 1)] = ns_split_pair(x[0][j] * f, x[1][j] * f, &lo);
                if constexpr (kLo) tile[1][lp + 8 * (j >> 1)][lc + 32 * (j & 1)] = lo;
            }
        }
        __syncthreads();
        if (r0 + 64 < end) load(r0 + 64);
        if (c0 + c >= a.C) continue;
        const long long at = ((long long)mat * a.C + c0 + c) * a.ld + r0 + 2 * rp;
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
            if (r0 + 2 * (rp + q) >= a.R) break;
            auto run = [&](int t) {
                return make_uint4(tile[t][rp + q][c], tile[t][rp + q + 1][c], tile[t][rp + q + 2][c], tile[t][rp + q + 3][c]);
            };
            *reinterpret_cast<uint4*>(a.hi + at + 2 * q) = run(0);
            if constexpr (kLo)
                if (a.lo) *reinterpret_cast<uint4*>(a.lo + at + 2 * q) = run(1);
        }
    }
}

// ---- the steps -----------------------------------------------------------------------------------------
enum NsMode { NS_GRAM = 0, NS_POLY, NS_APPLY };
// How the last step stores O: through TMA boxes as it stands or flipped, or by plain stores where its
// rows are not multiples of 16 bytes
enum NsOut { NS_O_BOX = 1, NS_O_BOX_FLIP, NS_O_PLAIN, NS_O_PLAIN_FLIP };

// Maps of A, B, X (two buffers), X's rounding error and O with boxes of 64 columns: 128 rows for operands
// along K and for the epilogue's boxes, 64 ("_t") for X as APPLY's second operand and for transposed boxes
struct NsMaps {
    CUtensorMap a, a_t, b, b_t, x[2], x_t[2], lo, o, o_t;
};

struct NsArgs {
    int m, n, N, steps;
    int mt, nt;                  // tile rows and columns of X
    int tri, full;               // tiles of A's upper triangle, and of X
    int parts, last_parts;       // CTAs that store a part of a tile: both of a pair, or in the last tile row
                                 // the first alone where the second's rows are past the edge
    int h, halves;               // matrices of a half group, half groups in flight (see ns_unit)
    int per_cycle, cycles, supers;
    int units;
    int k_gram, k_poly;          // K slices
    int ab_lo;                   // A and B keep their rounding errors: matrix N + i of their arrays, second products
    int first_lo;                // the first X has a rounding error (else it is exact)
    int out_kind;                // NsOut
    float co[3 * MOE_ORTHOGONALISE_MAX_STEPS];
    const float* inv_s;          // [N]
    int* done;                   // [N][1 + 2 mt] parts of tiles stored: GRAM's; POLY's and APPLY's by tile row
    __nv_bfloat16* O;
    int* status;
    long long wait_limit;
    int withhold_loads;
};

__device__ __forceinline__ void ns_wait_drain(uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kDrainCycles) break;
}

struct NsUnit {
    int mode, step, mat, i, j;
    bool valid;
};
// A matrix's phases GRAM, POLY, APPLY of each step follow one another: POLY starts when GRAM has stored every
// tile, APPLY of a tile row when POLY has stored that row of B (POLY goes by rows of the triangle, each of
// which completes one, by symmetry), GRAM of a tile when APPLY has stored its two rows of X.  What a phase
// writes while the one before still runs, that one no longer reads: POLY's tiles that touch a row of A are
// stored before that row of X, and so of A, can change.
// So that the CTAs have other work while a phase waits, and that X, A and B stay in L2 from one phase to the
// next, two half groups of h matrices are in flight, half a step apart: cycle c holds
//   GRAM(a) APPLY(b, the step before) POLY(a) GRAM(b) APPLY(a) POLY(b)
// with a, b the halves of group c / steps in step c % steps; a single matrix goes GRAM POLY APPLY.  CTAs take
// the units of this list in turn; every unit depends on earlier ones only.
__device__ __forceinline__ NsUnit ns_unit(int unit, const NsArgs& a) {
    NsUnit u;
    int c = unit / a.per_cycle, left = unit - c * a.per_cycle, b = 0;
    const int t = a.h * a.tri, f = a.h * a.full;
    if (a.halves == 1) {
        u.mode = left < t ? NS_GRAM : left < 2 * t ? NS_POLY : NS_APPLY;
        left -= u.mode * t;
    } else if (left < t) {
        u.mode = NS_GRAM;
    } else if ((left -= t) < f) {
        u.mode = NS_APPLY;
        b = 1;
        --c;
    } else if ((left -= f) < t) {
        u.mode = NS_POLY;
    } else if ((left -= t) < t) {
        u.mode = NS_GRAM;
        b = 1;
    } else if ((left -= t) < f) {
        u.mode = NS_APPLY;
    } else {
        left -= f;
        u.mode = NS_POLY;
        b = 1;
    }
    const int group = c / a.steps;
    u.step = c - group * a.steps;
    const int tiles = u.mode == NS_APPLY ? a.full : a.tri;
    const int k = left / tiles;
    left -= k * tiles;
    u.mat = group * a.halves * a.h + b * a.h + k;
    u.valid = c >= 0 && group < a.supers && u.mat < a.N;
    if (u.mode == NS_APPLY) {
        u.i = left / a.nt;
        u.j = left - u.i * a.nt;
    } else {   // the upper triangle by columns, column j having j + 1 tiles; by rows, the same backwards
        if (u.mode == NS_POLY) left = a.tri - 1 - left;
        int j = (int)((sqrtf(8.f * left + 1.f) - 1.f) * 0.5f);
        while (j * (j + 1) / 2 > left) --j;
        while ((j + 1) * (j + 2) / 2 <= left) ++j;
        u.i = left - j * (j + 1) / 2;
        u.j = j;
        if (u.mode == NS_POLY) {
            u.j = a.mt - 1 - u.i;
            u.i = a.mt - 1 - j;
        }
    }
    return u;
}
// The tile's columns, rounded up to what an MMA takes: a last tile column costs what it holds.
template <int TILE>
__device__ __forceinline__ int ns_width(const NsUnit& u, const NsArgs& a) {
    return min(TILE, ((u.mode == NS_APPLY ? a.n : a.m) - u.j * TILE + 31) & ~31);
}
// A pair's whole tile on the diagonal of A or B: its operands are the same rows, and one copy serves as both
// (256 x 768 x 2048: 1.1% less time; one CTA's tiles, whose phases wait for those off the diagonal, gain
// nothing: 3 x 1001 x 777 158.1 -> 159.8 us).
template <bool PAIR>
__device__ __forceinline__ bool ns_same(const NsUnit& u, int width) {
    return PAIR && u.mode != NS_APPLY && u.i == u.j && width == 256;
}
// The matrix's counters, and what they hold when a unit's inputs are stored.  A part is counted only after
// its accumulator has been stored, which its own inputs precede, so no count runs ahead of its phase.
__device__ __forceinline__ int* ns_count(const NsArgs& a, int mat) { return a.done + (long long)mat * (1 + 2 * a.mt); }
__device__ __forceinline__ int ns_row_parts(const NsArgs& a, int i) { return i + 1 < a.mt ? a.parts : a.last_parts; }
__device__ __forceinline__ bool ns_wait_count(const int* count, int need, volatile int* abort_flag, const NsArgs& a) {
    if (ld_acquire_gpu(count) >= need) return true;
    const long long t0 = clock64();
    while (ld_acquire_gpu(count) < need) {
        if (*abort_flag) return false;
        if (clock64() - t0 > a.wait_limit) {
            *abort_flag = 1;
            set_status(a.status, MOE_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool ns_wait_unit(const NsUnit& u, volatile int* abort_flag, const NsArgs& a) {
    const int* c = ns_count(a, u.mat);
    if (u.mode == NS_GRAM)
        return u.step == 0 ||
               (ns_wait_count(c + 1 + a.mt + u.i, u.step * a.nt * ns_row_parts(a, u.i), abort_flag, a) &&
                (u.i == u.j || ns_wait_count(c + 1 + a.mt + u.j, u.step * a.nt * ns_row_parts(a, u.j), abort_flag, a)));
    // of the triangle only the last diagonal tile is in the last tile row
    const int less = a.parts - a.last_parts;
    if (u.mode == NS_POLY) return ns_wait_count(c, (u.step + 1) * (a.tri * a.parts - less), abort_flag, a);
    // the mt tiles (i, i..) and (..i-1, i)
    return ns_wait_count(c + 1 + u.i, (u.step + 1) * (a.mt * a.parts - (u.i + 1 < a.mt ? 0 : less)), abort_flag, a);
}

// Chunk `at` (16 bytes) of row r of a box
__device__ __forceinline__ uint32_t ns_sw(int r, int at) { return (uint32_t)(r * 128 + ((at ^ (r & 7)) << 4)); }
// the thread's 32 columns of its row (columns 32 half .. of the box), packed in pairs
__device__ __forceinline__ void ns_box_read(uint32_t* v, uint32_t box, int r, int half) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 w = ld_shared_v4(box + ns_sw(r, 4 * half + q));
        v[4 * q] = w.x; v[4 * q + 1] = w.y; v[4 * q + 2] = w.z; v[4 * q + 3] = w.w;
    }
}
__device__ __forceinline__ void ns_box_row(uint32_t box, int r, int half, const uint32_t* v) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        st_shared_v4(box + ns_sw(r, 4 * half + q), make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
}
// the transpose, as two boxes of 64 rows x 64 columns: value j goes to row 32 half + j, column r mod 64 of
// box r / 64 (a warp writes 64 consecutive bytes at a time)
__device__ __forceinline__ void ns_box_col(uint32_t box, int r, int half, const uint32_t* v) {
    box += (r >> 6) * 8192 + (r & 7) * 2;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint16_t h = (uint16_t)(j & 1 ? v[j >> 1] >> 16 : v[j >> 1] & 0xffffu);
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(box + ns_sw(32 * half + j, (r & 63) >> 3)), "h"(h) : "memory");
    }
}

// What the epilogue side does with a unit's chunks of 64 columns.
struct NsPart {
    int row0, n0, chunks;      // the CTA's first row, the tile's first column
    int out_kind;              // NsOut in the last step's APPLY, else 0
    bool load;                 // POLY: the chunk of A comes in, and of its rounding error; APPLY: X's rounding error
    bool twin, keep_lo;        // out go the transpose as well, or a rounding error
};
template <int TILE>
__device__ __forceinline__ NsPart ns_part(const NsUnit& u, int rank, const NsArgs& a) {
    NsPart p;
    p.row0 = u.i * TILE + rank * 128;
    p.n0 = u.j * TILE;
    p.chunks = p.row0 < a.m ? (min(TILE, (u.mode == NS_APPLY ? a.n : a.m) - p.n0) + 63) / 64 : 0;
    p.out_kind = u.mode == NS_APPLY && u.step + 1 == a.steps ? a.out_kind : 0;
    // the last step reads X without its rounding error, so the step before keeps none
    p.load = u.mode == NS_POLY || (u.mode == NS_APPLY && u.step + 1 < a.steps && (u.step > 0 || a.first_lo));
    p.keep_lo = u.mode == NS_APPLY ? u.step + 2 < a.steps : a.ab_lo;
    p.twin = u.mode != NS_APPLY && u.i != u.j;
    return p;
}

// What the epilogue multiplies: the accumulator; in POLY the tile of A that came with it, by an fp16 pair whose
// sum is b to 22 bits, and a goes to B's diagonal; in APPLY X's rounding error; and in the first step the whole
// by the rest of the norm.  The scales of X, A, B and O are in there.
struct NsFactors {
    float d, is, diag;
    uint32_t hi, lo, half;
};
__device__ __forceinline__ NsFactors ns_factors(const NsUnit& u, const NsPart& p, const NsArgs& a) {
    NsFactors f;
    f.is = u.step == 0 ? __ldg(a.inv_s + u.mat) : 1.f;
    f.d = u.mode == NS_GRAM   ? kABScale / (kXScale * kXScale) * f.is * f.is
          : u.mode == NS_POLY ? a.co[3 * u.step + 2] / kABScale
                              : (p.out_kind ? 1.f / kXScale : 1.f) / kABScale;
    f.diag = a.co[3 * u.step] * kABScale;
    const float x = u.mode == NS_POLY ? a.co[3 * u.step + 1] : a.co[3 * u.step] / kLoScale;
    f.hi = ns_pack_half(x, 0.f);
    f.lo = ns_pack_half(x - ns_unpack_half(f.hi).x, 0.f);
    f.half = ns_pack_half(0.5f * x, 0.f);   // (A's rounding error is held twice)
    return f;
}

// Every step of every matrix in one launch of persistent CTAs, a warp to each job, all waits bounded:
//   warp 0      operand K slices by TMA into a ring of four stages of 32 KB
//   warp 1      MMAs into one of two accumulators
//   warps 2-9   epilogue: lane quarter w % 4, alternate 32 columns; a chunk is 64 columns of the tile
//   warp 10     watches the matrices' counters ahead of the others: `ready` units of this CTA have inputs
//   warp 11     what a chunk needs besides its accumulator (POLY: A; APPLY: X's rounding error), by
//               TMA into one of three slots
//   warp 12     stores the slot, where the epilogue has put the results in their place, frees it, and
//               counts the tile once its stores are complete
// The box loads and stores have threads of their own since an epilogue warp that issued them spent more
// time there than on its arithmetic, and boxes of 128-byte rows since narrower ones kept the TMA busy
// (12,600 cycles a tile of APPLY at K = 768, against 7,900 for its MMAs).
//   PAIR: two CTAs share a 256 x 256 tile (cta_group::2), each holding 128 rows of the first operand and
//   half of the second; otherwise one CTA computes 128 x 128.
// GRAM and POLY are symmetric: tiles of the upper triangle alone, and those above the diagonal are stored
// twice, as they are and transposed through shared memory.  Operands: GRAM rows of X by rows of X, POLY
// rows of A by rows of A (A = A^T), both contiguous along K; APPLY rows of B by columns of X (contiguous
// along N).  The TMA fills K past the edge with zeros and drops stores outside a matrix, so no size needs
// padding beyond 16-byte rows.
template <bool PAIR>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_steps_kernel(const __grid_constant__ NsMaps maps, const __grid_constant__ NsArgs a) {
    grid_dep_wait();
    constexpr int kTile = PAIR ? 256 : 128;      // rows and columns of a unit's tile
    constexpr int kOperand = 128 * 128;          // bytes of one operand's K slice per CTA: 128 x 64 fp16
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + kNsStages * kOperand;
    uint8_t* sBox = sB + kNsStages * kOperand;
    uint64_t* full = reinterpret_cast<uint64_t*>(sBox + kNsSlots * 2 * kNsBox);
    uint64_t* empty = full + kNsStages;
    uint64_t* tfull = empty + kNsStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* box_full = drain + 1;              // a slot's loads have landed,
    uint64_t* box_done = box_full + kNsSlots;    // its results are written,
    uint64_t* box_free = box_done + kNsSlots;    // and stored
    uint32_t* tslot = reinterpret_cast<uint32_t*>(box_free + kNsSlots);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* ready = reinterpret_cast<int*>(tslot + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int unit0 = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int stride = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kNsStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull + b, 1);
            mbar_init(tempty + b, (PAIR ? 2 : 1) * kNsEpi);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < kNsSlots; ++i) {
            mbar_init(box_full + i, 1);
            mbar_init(box_done + i, kNsEpi);
            mbar_init(box_free + i, 1);
        }
        *abort_flag = 0;
        *ready = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (PAIR) tmem_alloc_pair(tslot, 2 * kTile);
        else tmem_alloc(tslot, 2 * kTile);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // the peer's barriers exist before any copy or commit reaches them
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // until this CTA's unit q has its inputs (false: gave up); then this thread's TMA loads may read them
    auto inputs = [&](int q) {
        if (ld_acquire_cta_shared(ready) <= q) {
            const long long t0 = clock64();
            while (ld_acquire_cta_shared(ready) <= q) {
                if (*abort_flag) return false;
                if (clock64() - t0 > a.wait_limit) {
                    *abort_flag = 1;
                    set_status(a.status, MOE_DEV_TIMEOUT);
                    return false;
                }
            }
        }
        fence_proxy_async_global();
        return true;
    };

    if (warp == 0) {
        if (lane == 0 && !a.withhold_loads) {
            int stage = 0, q = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int unit = unit0; unit < a.units && ok; unit += stride, ++q) {
                const NsUnit t = ns_unit(unit, a);
                if (!t.valid) continue;
                if (!inputs(q)) break;
                const int width = ns_width<kTile>(t, a);
                const int m0 = t.i * kTile + rank * 128, n0 = t.j * kTile + rank * (width / 2);
                const bool apply = t.mode == NS_APPLY;
                const CUtensorMap* tmA = t.mode == NS_GRAM ? &maps.x[t.step & 1] : apply ? &maps.b : &maps.a;
                const CUtensorMap* tmB = apply ? &maps.x_t[t.step & 1] : tmA;
                const int wrap = t.mode == NS_GRAM ? a.k_gram : a.k_poly;
                const bool same = ns_same<PAIR>(t, width);
                const uint32_t bytes = (PAIR ? 2 : 1) * (same ? kOperand : 2 * kOperand);
                const int k_blocks = t.mode != NS_GRAM && a.ab_lo ? 2 * wrap : wrap;   // A A, A by its error; B X, its error by X
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!mbar_wait(empty + stage, phase ^ 1u, abort_flag, a.status, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dA = sA + stage * kOperand;
                    uint8_t* dB = sB + stage * kOperand;
                    const bool second = kb >= wrap;
                    const int k0 = (second ? kb - wrap : kb) * 64;
                    const int matA = second && apply ? t.mat + a.N : t.mat, matB = second && !apply ? t.mat + a.N : t.mat;
                    if constexpr (PAIR) {
                        // both CTAs' copies land on the leader's barrier, which expects both
                        const uint32_t lbar = cluster_addr(full + stage, 0);
                        if (rank == 0) mbar_arrive_expect_tx(full + stage, bytes);
                        tma_load_3d_pair(dA, tmA, lbar, k0, m0, matA);
                        if (apply) {
                            tma_load_3d_pair(dB, tmB, lbar, n0, k0, t.mat);
                            tma_load_3d_pair(dB + kOperand / 2, tmB, lbar, n0 + 64, k0, t.mat);
                        } else if (!same) {
                            tma_load_3d_pair(dB, tmB, lbar, k0, n0, matB);
                        }
                    } else {
                        mbar_arrive_expect_tx(full + stage, bytes);
                        tma_load_3d(dA, tmA, full + stage, k0, m0, matA);
                        if (apply) {
                            tma_load_3d(dB, tmB, full + stage, n0, k0, t.mat);
                            tma_load_3d(dB + kOperand / 2, tmB, full + stage, n0 + 64, k0, t.mat);
                        } else if (!same) {
                            tma_load_3d(dB, tmB, full + stage, k0, n0, matB);
                        }
                    }
                    ++issued;
                    if (++stage == kNsStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // this CTA's copies have landed (bounded) before it exits, whoever gave up; a pair's land on
            // the leader's barriers, and the peer waits for the releases that follow them instead
            uint64_t* last = rank == 0 ? full : empty;
            for (int s = 0; s < kNsStages; ++s)
                if (issued > s) ns_wait_drain(last + s, (uint32_t)(((issued - s + kNsStages - 1) / kNsStages - 1) & 1));
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            long long consumed = 0;
            bool ok = true;
            const uint32_t a_base = smem_u32(sA), b_base = smem_u32(sB);
            for (int unit = unit0; unit < a.units && ok; unit += stride) {
                const NsUnit t = ns_unit(unit, a);
                if (!t.valid) continue;
                const bool apply = t.mode == NS_APPLY;
                const int k_blocks = t.mode == NS_GRAM ? a.k_gram : a.ab_lo ? 2 * a.k_poly : a.k_poly;
                if (!(PAIR ? mbar_wait_cluster(tempty + acc, acc_phase ^ 1u, abort_flag, a.status, a.wait_limit)
                           : mbar_wait(tempty + acc, acc_phase ^ 1u, abort_flag, a.status, a.wait_limit))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * kTile);
                const int width = ns_width<kTile>(t, a);
                const uint32_t idesc = idesc_f16(kTile, width, false, apply);
                const uint32_t other = ns_same<PAIR>(t, width) ? a_base : b_base;
                const uint32_t b_step = apply ? 2048 : 32, b_lbo = apply ? kOperand / 2 : 16;
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!mbar_wait(full + stage, phase, abort_flag, a.status, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = a_base + stage * kOperand, sb = other + stage * kOperand;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = sdesc_sw128(sa + ks * 32, 16, 1024);
                        const uint64_t bd = sdesc_sw128(sb + ks * b_step, b_lbo, 1024);
                        if constexpr (PAIR) mma_bf16_pair(d, ad, bd, idesc, (kb | ks) != 0);
                        else mma_bf16(d, ad, bd, idesc, (kb | ks) != 0);
                    }
                    if constexpr (PAIR) mma_commit_pair_mc(empty + stage, 0x3);
                    else mma_commit(empty + stage);
                    ++consumed;
                    if (++stage == kNsStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if constexpr (PAIR) mma_commit_pair_mc(tfull + acc, 0x3);
                else mma_commit(tfull + acc);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok) {
                if constexpr (PAIR) mma_commit_pair_mc(drain, 0x1);
                else mma_commit(drain);
                ns_wait_drain(drain, 0);
            } else if (PAIR) {
                // the releases of the last stages have landed before the CTA may exit
                for (int s = 0; s < kNsStages; ++s)
                    if (consumed > s)
                        ns_wait_drain(empty + s, (uint32_t)(((consumed - s + kNsStages - 1) / kNsStages - 1) & 1));
            }
        }
    } else if (warp == 2 + kNsEpi) {
        if (lane == 0) {
            int q = 0;
            bool ok = true;
            for (int unit = unit0; unit < a.units && ok; unit += stride, ++q) {
                const NsUnit t = ns_unit(unit, a);
                ok = !t.valid || ns_wait_unit(t, abort_flag, a);
                if (ok) st_release_cta_shared(ready, q + 1);
            }
        }
    } else if (warp == 3 + kNsEpi) {
        if (lane == 0 && !a.withhold_loads) {
            uint32_t k = 0;   // chunks so far; slot: mod kNsSlots
            int q = 0;
            bool ok = true;
            for (int unit = unit0; unit < a.units && ok; unit += stride, ++q) {
                const NsUnit t = ns_unit(unit, a);
                if (!t.valid) continue;
                const NsPart p = ns_part<kTile>(t, rank, a);
                if (p.chunks == 0) continue;
                if (p.load && !inputs(q)) break;
                const CUtensorMap* tm = t.mode == NS_POLY ? &maps.a : &maps.lo;
                const bool poly = t.mode == NS_POLY, both = poly && a.ab_lo;   // A, and its rounding error (twice)
                const int second = poly ? 0 : kNsBox;   // the rounding error's place in the slot
                for (int c = 0; c < p.chunks; ++c, ++k) {
                    const int slot = k % kNsSlots;
                    if (!mbar_wait(box_free + slot, (k / kNsSlots & 1) ^ 1u, abort_flag, a.status, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    if (!p.load) {
                        mbar_arrive(box_full + slot);
                        continue;
                    }
                    uint8_t* box = sBox + slot * 2 * kNsBox;
                    mbar_arrive_expect_tx(box_full + slot, both ? 2 * kNsBox : kNsBox);
                    tma_load_3d(box + second, tm, box_full + slot, p.n0 + 64 * c, p.row0, t.mat);
                    if (both) tma_load_3d(box + kNsBox, tm, box_full + slot, p.n0 + 64 * c, p.row0, t.mat + a.N);
                }
            }
            // every load has landed (bounded) before the CTA exits
            for (uint32_t i = k > kNsSlots ? k - kNsSlots : 0; i < k; ++i)
                ns_wait_drain(box_full + i % kNsSlots, i / kNsSlots & 1);
        }
    } else if (warp == 4 + kNsEpi) {
        if (lane == 0) {
            uint32_t k = 0;
            bool ok = true;
            for (int unit = unit0; unit < a.units && ok; unit += stride) {
                const NsUnit t = ns_unit(unit, a);
                if (!t.valid) continue;
                const NsPart p = ns_part<kTile>(t, rank, a);
                const CUtensorMap* tm = t.mode == NS_GRAM ? &maps.a : t.mode == NS_POLY ? &maps.b
                                        : p.out_kind      ? &maps.o : &maps.x[1 - (t.step & 1)];
                const CUtensorMap* tm_t = t.mode == NS_GRAM ? &maps.a_t : t.mode == NS_POLY ? &maps.b_t : &maps.o_t;
                for (int c = 0; c < p.chunks; ++c, ++k) {
                    const int slot = k % kNsSlots, col = p.n0 + 64 * c;
                    uint8_t* box = sBox + slot * 2 * kNsBox;
                    if (!mbar_wait(box_done + slot, k / kNsSlots & 1, abort_flag, a.status, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    if (p.out_kind < NS_O_BOX_FLIP) tma_store_3d(tm, box, col, p.row0, t.mat);
                    if (p.twin || p.out_kind == NS_O_BOX_FLIP) {
                        tma_store_3d(tm_t, box + kNsBox, p.row0, col, t.mat);
                        if (p.row0 + 64 < a.m) tma_store_3d(tm_t, box + kNsBox + 8192, p.row0 + 64, col, t.mat);
                    } else if (p.keep_lo) {
                        if (t.mode == NS_APPLY) tma_store_3d(&maps.lo, box + kNsBox, col, p.row0, t.mat);
                        else tma_store_3d(tm, box + kNsBox, col, p.row0, t.mat + a.N);
                    }
                    bulk_commit();
                    if (c > 0) {   // the slot before this one has been read
                        bulk_wait_read<1>();
                        mbar_arrive(box_free + (k - 1) % kNsSlots);
                    }
                }
                if (!ok) break;
                if (p.chunks == 0) continue;   // not counted: it would be before its turn
                bulk_wait_read<0>();
                mbar_arrive(box_free + (k - 1) % kNsSlots);
                if (!p.out_kind) {
                    // this CTA's part of the tile is stored, and visible to whoever sees the count
                    bulk_wait_all();
                    fence_proxy_async_global();
                    int* count = ns_count(a, t.mat);
                    if (t.mode == NS_GRAM) {
                        red_release_gpu_add(count, 1);
                    } else if (t.mode == NS_POLY) {
                        red_release_gpu_add(count + 1 + t.i, 1);
                        if (t.i != t.j) red_release_gpu_add(count + 1 + t.j, 1);
                    } else {
                        red_release_gpu_add(count + 1 + a.mt + t.i, 1);
                    }
                }
            }
            bulk_wait_all();   // the stores are complete before the CTA exits
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const int br = quarter * 32 + lane;      // row of the CTA's tile, and of a box
        uint32_t k = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int unit = unit0; unit < a.units && ok; unit += stride) {
            const NsUnit t = ns_unit(unit, a);
            if (!t.valid) continue;
            const NsPart p = ns_part<kTile>(t, rank, a);
            const NsFactors f = ns_factors(t, p, a);
            if (!__all_sync(0xffffffffu, mbar_wait(tfull + acc, acc_phase, abort_flag, a.status, a.wait_limit))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < p.chunks; ++c, ++k) {
                const int slot = k % kNsSlots, col = p.n0 + 64 * c + 32 * half;
                const uint32_t sbox = smem_u32(sBox + slot * 2 * kNsBox);
                float v[32];
                uint32_t out[16], low[16];
                tmem_ld32(tmem + lane_addr + (uint32_t)(acc * kTile + 64 * c + 32 * half), v);
                ok = __all_sync(0xffffffffu,
                                mbar_wait(box_full + slot, k / kNsSlots & 1, abort_flag, a.status, a.wait_limit));
                if (!ok) break;
                if (t.mode == NS_GRAM && !p.keep_lo) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = ns_pack_half(v[2 * j] * f.d, v[2 * j + 1] * f.d);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= f.d;
                    if (t.mode == NS_POLY) {
                        ns_box_read(out, sbox, br, half);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            fma_f16x2(v + 2 * j, out[j], f.hi);
                            fma_f16x2(v + 2 * j, out[j], f.lo);
                        }
                        if (p.keep_lo) {
                            ns_box_read(low, sbox + kNsBox, br, half);
#pragma unroll
                            for (int j = 0; j < 16; ++j) fma_f16x2(v + 2 * j, low[j], f.half);
                        }
                        if (p.row0 + 32 * quarter == col) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j == lane) v[j] += f.diag;
                        }
                    } else if (p.load) {
                        ns_box_read(low, sbox + kNsBox, br, half);
#pragma unroll
                        for (int j = 0; j < 16; ++j) fma_f16x2(v + 2 * j, low[j], f.hi);
                    }
                    if (t.step == 0 && t.mode == NS_APPLY) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= f.is;
                    }
                    if (p.out_kind) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) out[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) out[j] = ns_pack_half(v[2 * j], v[2 * j + 1]);
                        if (p.keep_lo) {
                            const uint32_t minus = ns_pack_half(-1.f, 0.f);
                            const float scale = t.mode == NS_GRAM ? 2.f : t.mode == NS_POLY ? 1.f : kLoScale;
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                fma_f16x2(v + 2 * j, out[j], minus);
                                low[j] = ns_pack_half(v[2 * j] * scale, v[2 * j + 1] * scale);
                            }
                        }
                    }
                }
                // results replace what this thread read; transposes go to the second box, which then holds
                // nothing that another warp still reads
                if (p.out_kind == NS_O_PLAIN_FLIP) {   // a warp's 32 rows are 64 consecutive bytes of O
                    const int r = p.row0 + br;
                    if (r < a.m) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < a.n)
                                reinterpret_cast<uint16_t*>(a.O)[((long long)t.mat * a.n + col + j) * a.m + r] =
                                    (uint16_t)(j & 1 ? out[j >> 1] >> 16 : out[j >> 1]);
                    }
                } else if (p.out_kind == NS_O_BOX_FLIP) {
                    ns_box_col(sbox + kNsBox, br, half, out);
                } else {
                    ns_box_row(sbox, br, half, out);
                    if (p.twin) ns_box_col(sbox + kNsBox, br, half, out);
                    else if (p.keep_lo) ns_box_row(sbox + kNsBox, br, half, low);
                }
                if (p.out_kind == NS_O_PLAIN) {   // 64 consecutive bytes of a row of O at a time
                    __syncwarp();
                    const int r0 = p.row0 + 32 * quarter;
                    if (col + lane < a.n)
                        for (int q = 0; q < min(32, a.m - r0); ++q) {
                            uint16_t h;
                            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h)
                                         : "r"(sbox + ns_sw(32 * quarter + q, 4 * half + (lane >> 3)) + (lane & 7) * 2)
                                         : "memory");
                            reinterpret_cast<uint16_t*>(a.O)[((long long)t.mat * a.m + r0 + q) * a.n + col + lane] = h;
                        }
                }
                fence_proxy_async_cta();
                __syncwarp();
                if (lane == 0) mbar_arrive(box_done + slot);
            }
            tc_fence_before();
            __syncwarp();
            if (!ok) break;
            if (lane == 0) {
                if (PAIR && rank == 1) mbar_arrive_cluster(tempty + acc, 0);
                else mbar_arrive(tempty + acc);
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // no commit or release from the peer is still in flight
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, 2 * kTile);
        else tmem_dealloc(tmem, 2 * kTile);
    }
}

// ---- matrices of up to 8 rows: fp32 throughout ------------------------------------------------------------
// With so few singular values the rounding errors of fp16 operands do not average out (1 x 3 and 5 x 2 came out
// up to 0.53 % off), and the work is small: a CTA takes a matrix, keeps the product M of the steps' a I + B,
// 8 x 8, and forms X = M G / (|G| + eps) a column at a time, once a step for A = X X^T and once for O (a
// recursion of A alone would need no more than the first of these passes, but it loses what is below A's
// rounding, and with it that A has no negative eigenvalue).  Over 1024 columns a cluster of up to eight CTAs
// takes the matrix, each some of its columns and all the sums.  Latency of the passes and of six block sums binds it
// (40 x 8 x 70: 13.8 us, 8 x 32768: 45 us; on the tensor cores, by the kernel below, 20.7 and 86).
constexpr int kTinyRows = 8;
constexpr int kTinyThreads = 512;
struct NsTiny {
    int m, n, flip, steps, ctas;
    float eps;
    float co[3 * MOE_ORTHOGONALISE_MAX_STEPS];
};
// element (i, k), i <= k, of a symmetric 8 x 8 matrix among its 36
__device__ __forceinline__ constexpr int ns_tri(int i, int k) { return i * (2 * kTinyRows - 1 - i) / 2 + k; }

template <typename T>
__global__ void __launch_bounds__(kTinyThreads) ns_tiny_kernel(const T* G, __nv_bfloat16* O, const NsTiny a) {
    grid_dep_wait();
    constexpr int K = kTinyRows, kTri = K * (K + 1) / 2, kWarps = kTinyThreads / 32;
    __shared__ float part[kWarps][kTri], sums[2][kTri], sA[K][K], sC[K][K], sM[K][K];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ti = threadIdx.x >> 3, tk = threadIdx.x & 7;
    const int S = a.ctas, j0 = (int)(blockIdx.x % S) * kTinyThreads + threadIdx.x;
    const long long base = (long long)(blockIdx.x / S) * a.m * a.n;
    const int si = a.flip ? 1 : a.n, sj = a.flip ? a.m : 1;
    float M[K][K];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) M[i][k] = i == k ? 1.f : 0.f;
    if (threadIdx.x < K * K) sM[ti][tk] = ti == tk ? 1.f : 0.f;
    float f = 1.f;   // 1 / (|G| + eps), which the first pass finds
    auto column = [&](int j, float* x) {
        float g[K];
#pragma unroll
        for (int i = 0; i < K; ++i) g[i] = ns_val(G, base + (long long)min(i, a.m - 1) * si + (long long)j * sj);
#pragma unroll
        for (int i = 0; i < K; ++i) g[i] = i < a.m ? g[i] * f : 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            x[i] = M[i][0] * g[0];
#pragma unroll
            for (int k = 1; k < K; ++k) x[i] += M[i][k] * g[k];
        }
    };
    for (int s = 0; s < a.steps; ++s) {
        float sum[kTri], x[K];
#pragma unroll
        for (int e = 0; e < kTri; ++e) sum[e] = 0.f;
        for (int j = j0; j < a.n; j += S * kTinyThreads) {
            column(j, x);
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int k = i; k < K; ++k) sum[ns_tri(i, k)] += x[i] * x[k];
        }
#pragma unroll
        for (int e = 0; e < kTri; ++e) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
            if (lane == 0) part[warp][e] = sum[e];
        }
        __syncthreads();
        float* mine = sums[s & 1];   // (read by the others until they have passed the next step's barrier)
        if (threadIdx.x < kTri) {
            float v = 0.f;
            for (int w = 0; w < kWarps; ++w) v += part[w][threadIdx.x];
            mine[threadIdx.x] = v;
        }
        if (S > 1) cluster_sync();
        else __syncthreads();
        auto total = [&](int e) {
            float v = S > 1 ? 0.f : mine[e];
            if (S > 1)
                for (int c = 0; c < S; ++c) v += ld_cluster_f32(cluster_addr(mine + e, c));
            return v;
        };
        if (threadIdx.x < K * K) sA[ti][tk] = total(ns_tri(min(ti, tk), max(ti, tk)));
        __syncthreads();
        if (s == 0) {
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i) sq += sA[i][i];
            const float norm = sqrtf(sq);
            f = norm <= 3.4e38f ? 1.f / (norm + a.eps) : NAN;
            __syncthreads();
            if (threadIdx.x < K * K) sA[ti][tk] = sA[ti][tk] * f * f;
        }
        __syncthreads();
        if (threadIdx.x < K * K) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < K; ++q) v += sA[ti][q] * sA[q][tk];
            sC[ti][tk] = (ti == tk ? a.co[3 * s] : 0.f) + a.co[3 * s + 1] * sA[ti][tk] + a.co[3 * s + 2] * v;
        }
        __syncthreads();
        float v = 0.f;
        if (threadIdx.x < K * K)
#pragma unroll
            for (int q = 0; q < K; ++q) v += sC[ti][q] * sM[q][tk];
        __syncthreads();
        if (threadIdx.x < K * K) sM[ti][tk] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int k = 0; k < K; ++k) M[i][k] = sM[i][k];
    }
    for (int j = j0; j < a.n; j += S * kTinyThreads) {   // O may be G: a column is read before it is written
        float x[K];
        column(j, x);
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < a.m) O[base + (long long)i * si + (long long)j * sj] = __float2bfloat16_rn(x[i]);
    }
    if (S > 1) cluster_sync();   // no CTA's sums are read any more
}

// ---- matrices of up to 128 rows: the whole operator in one kernel --------------------------------------
// The products of a matrix with m <= 128 are too small to be launches of their own (17 of them took
// 120 us at 128 x 2048).  A cluster of CTAs takes a matrix, each CTA 256 of its columns, from G to O: X in
// fp32 registers (a thread has a row's 128 columns) and its fp16 copy in shared memory, where the rows of
// 64 columns that GRAM reads along K are, unchanged, what APPLY reads along N.  Per step:
//   partial A over the CTA's columns -> the cluster's sum, each CTA adding the rows it owns in the CTAs'
//   order and sending them to all as fp16 -> A A and B in every CTA -> X of the CTA's columns.
// Where m leaves room, up to eight blocks of 256 columns lie one below the other in the CTA's 128 rows: A is
// the sum of the diagonal blocks of their product, and with A and B laid out block-diagonally the rest goes
// as before, with as many CTAs less (96 matrices of 20 x 1210: 80 us; 100 take 202 with the large kernels).
// A's rounding error lies below A in each chunk of columns, so that A A and A by its error are one MMA of 256 columns
// (of 128 each, with operands that differ, an MMA takes 112 cycles, and 16 of them 300 more than these eight).  The
// errors of A and B cost 16 x 128 x 256 24.6 -> 31.8 us and 1 x 128 x 2048 47.9 -> 55.9.
constexpr int kSmallX = 4 * 16384;   // X: four chunks of 128 rows x 64 columns (128-byte swizzle)
// A, and later B, with its rounding error: for each 64 columns the 128 rows of A and then those of its error
constexpr int kSmallA = 4 * 16384, kSmallLo = 16384, kSmallChunk = 2 * 16384;
constexpr int kSmallBytes = 1024 + kSmallX + 2 * kSmallA + 256;   // X, A, and the partial A in fp32, later B

struct NsSmall {
    int R, C, m, n, mp, log_mp, log_ctas, steps, flip;   // mp: rows of a block, 128 / mp blocks one below the other
    float eps;
    float co[3 * MOE_ORTHOGONALISE_MAX_STEPS];
    __nv_bfloat16* O;
    int* status;
    long long wait_limit;
    int withhold;
};

template <int W, int STEP, int UNROLL>
__device__ __forceinline__ void ns_stage_in(uint32_t to, const void* from, int bytes) {
    const NsWords<W> words(reinterpret_cast<uintptr_t>(from), bytes);
    words.template each<STEP, UNROLL>(threadIdx.x & (STEP - 1), [&](int w, int held) {
        if constexpr (W == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + w), "l"(words.at + w), "r"(held) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + w), "l"(words.at + w), "r"(held) : "memory");
    });
}
__device__ __forceinline__ uint16_t ns_lds16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ns_lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
// a run of bf16: the whole words, then (flip's first and last thread, or a row's lanes) what is before and after
template <int W, int STEP>
__device__ __forceinline__ void ns_stage_out(void* to, uint32_t from, int bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(to) & ~uintptr_t(W - 1);
    const int begin = (int)(reinterpret_cast<uintptr_t>(to) - at), end = begin + bytes;
    const int lo = (begin + W - 1) & ~(W - 1), hi = end & ~(W - 1), t = threadIdx.x & (STEP - 1);
    if constexpr (W == 16) {
#pragma unroll 4
        for (int w = lo + W * t; w < hi; w += W * STEP) *reinterpret_cast<uint4*>(at + w) = ld_shared_v4(from + w);
    } else {   // up to 129 words
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lo + W * (t + k * STEP) < hi) v[k] = ns_lds32(from + lo + W * (t + k * STEP));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lo + W * (t + k * STEP) < hi) *reinterpret_cast<uint32_t*>(at + lo + W * (t + k * STEP)) = v[k];
    }
    const int head = begin + 2 * t, tail = max(hi, lo) + 2 * t;   // (a run within one word: lo > hi, all of it is head)
    if (head < min(lo, end)) *reinterpret_cast<uint16_t*>(at + head) = ns_lds16(from + head);
    if (tail < end) *reinterpret_cast<uint16_t*>(at + tail) = ns_lds16(from + tail);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kSmallThreads, 1) ns_small_kernel(const T* __restrict__ G, const NsSmall a) {
    grid_dep_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sX = smem;
    uint8_t* sA = sX + kSmallX;
    uint8_t* sP = sA + kSmallA;                 // fp32 [128][128], then B (fp16) and its rounding error
    uint64_t* done = reinterpret_cast<uint64_t*>(sP + kSmallA);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    float* warp_sums = reinterpret_cast<float*>(tslot + 2);   // [8]
    float* my_sum = warp_sums + 8;
    volatile int* open = reinterpret_cast<volatile int*>(warp_sums + 9);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = (int)gridDim.x, rank = S > 1 ? (int)cluster_ctarank() : 0, mat = blockIdx.y;
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane;                      // the thread's row in shared memory,
    const int mp = a.mp, blocks = 128 >> a.log_mp;
    const int i = row & (mp - 1);                             // of X,
    const int col0 = (rank * blocks + (row >> a.log_mp)) * kSmallCols + half * 128;   // and the first of its 128 columns
    if (threadIdx.x == 0) {
        mbar_init(done, 1);
        *abort_flag = 0;
        *open = -1;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    auto zero_a = [&] {   // A is zero outside its diagonal blocks
        for (int e = threadIdx.x; e < kSmallA / 16; e += kSmallThreads) st_shared_v4(smem_u32(sA) + 16 * e, make_uint4(0, 0, 0, 0));
    };
    if (VEC && blocks > 1) zero_a();
    float x[128];
    float sq = 0.f;
    const T* g = G + (long long)mat * a.R * a.C;
    const int block = row >> a.log_mp, left = i < a.m ? a.n - col0 : 0;   // columns that hold X
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
            if (i < a.m && col0 + j < a.n) {
                ns_val8(x + j, g + (long long)i * a.n + col0 + j);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) x[j + q] = 0.f;
            }
        }
    } else {
        constexpr int kBytes = (int)sizeof(T), kPitch = kSmallCols * kBytes + 4;
        const uint32_t stage = smem_u32(smem);
        const NsSlab slab{a.m, a.n, a.log_mp, a.flip, rank * blocks * kSmallCols};
        slab.each(kPitch, warp, [&](const NsRun& run) {
            if (a.flip) ns_stage_in<16, kSmallThreads, 4>(stage, g + run.first, run.count * kBytes);
            else ns_stage_in<4, 32, kPitch / 128>(stage + run.at, g + run.first, run.count * kBytes);
        });
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        // the thread's elements: every m-th of the CTA's run, or consecutive ones of its row's
        const uint32_t past = (uint32_t)reinterpret_cast<uintptr_t>(g + (a.flip ? slab.cta0 * a.m : i * a.n + slab.cta0));
        const uint32_t from = a.flip ? stage + (past & 15) + (uint32_t)(((block * kSmallCols + half * 128) * a.m + i) * kBytes)
                                     : stage + (past & 3) + (uint32_t)(row * kPitch + half * 128 * kBytes);
        const uint32_t step = a.flip ? a.m * kBytes : kBytes;
#pragma unroll
        for (int j = 0; j < 128; ++j) {   // (what is read past X is within the buffer, and dropped)
            float v;
            if constexpr (kBytes == 4) v = __uint_as_float(ns_lds32(from + j * step));
            else v = __uint_as_float((uint32_t)ns_lds16(from + j * step) << 16);
            x[j] = j < left ? v : 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < 128; j += 8) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += x[j + q] * x[j + q];
        sq += s;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) warp_sums[warp] = sq;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    if (!VEC && blocks > 1) zero_a();
    sq = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sq += warp_sums[w];
    if (S > 1) {
        if (threadIdx.x == 0) *my_sum = sq;
        cluster_sync();
        float part[16];
#pragma unroll
        for (int b = 0; b < 16; ++b) part[b] = b < S ? ld_cluster_f32(cluster_addr(my_sum, b)) : 0.f;
        sq = 0.f;
#pragma unroll
        for (int b = 0; b < 16; ++b) sq += part[b];
    }
    float is;
    const float f = ns_split(sqrtf(sq), a.eps, &is) * kXScale;
#pragma unroll
    for (int j = 0; j < 128; ++j) x[j] *= f;

    const uint32_t bX = smem_u32(sX), bA = smem_u32(sA), bP = smem_u32(sP);
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t tA = tmem, tX = tmem + 256;   // (A A too goes to tX)
    const int kx = min(4, max(0, (a.n - rank * blocks * kSmallCols + 63) / 64));   // chunks of X that hold columns
    const int km = blocks > 1 ? 8 : (a.m + 15) / 16;                      // MMA steps along the rows
    constexpr uint32_t kIdM = idesc_f16(128, 128, false, false), kIdP = idesc_f16(128, 256, false, false), kIdX = idesc_f16(128, 256, false, true);
    uint32_t phase = 0;
    // Every thread after its product's commit; on a wait that ran out the rest goes through without waiting, so that
    // the CTAs of a cluster stay in step, and without products: the one whose wait ran out is the only one that can
    // still be at work, and its commit ends `done`'s phase `open`.
    auto issues = [&] { return threadIdx.x == 0 && !a.withhold && !*abort_flag; };
    auto commit = [&] {
        mma_commit(done);
        *open = (int)phase;
    };
    auto wait_mma = [&] {
        mbar_wait(done, phase, abort_flag, a.status, a.wait_limit);
        phase ^= 1u;
        __syncwarp();
        tc_fence_after();
    };
    // X as fp16.  The last step takes a X from it too: with B and a of opposite signs by then, (a + B) of one X
    // errs less than a of the exact and B of the rounded (16 x 27: 1.73e-3 against 1.84e-3 before the rounding
    // to bf16; dropped from the step before it would cost matrices of low rank 2.3e-3 against 1.2e-3).
    auto put_x = [&](bool last) {
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
            uint32_t h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = ns_pack_half(x[j + 2 * q], x[j + 2 * q + 1]);
            st_shared_v4(bX + (2 * half + j / 64) * 16384 + ns_sw(row, (j & 63) >> 3), make_uint4(h[0], h[1], h[2], h[3]));
            if (last) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 r = ns_unpack_half(h[q]);
                    x[j + 2 * q] = r.x;
                    x[j + 2 * q + 1] = r.y;
                }
            }
        }
    };
    put_x(false);
    for (int s = 0; s < a.steps; ++s) {
        const float ca = a.co[3 * s], cb = a.co[3 * s + 1], fp = a.co[3 * s + 2] / kABScale;
        const uint32_t b_hi = ns_pack_half(cb, 0.f), b_lo = ns_pack_half(cb - ns_unpack_half(b_hi).x, 0.f),
                       b_half = ns_pack_half(0.5f * cb, 0.f);   // b to 22 bits, and half of it
        const float fa = kABScale / (kXScale * kXScale) * is * is, fx = is * ca, fv = is * (1.f / kABScale);
        fence_proxy_async_cta();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (issues()) {
            for (int c = 0; c < kx; ++c)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t d = sdesc_sw128(bX + c * 16384 + ks * 32, 16, 1024);
                    mma_bf16(tA, d, d, kIdM, (c | ks) != 0);
                }
            commit();
        }
        wait_mma();
        if (S == 1 && blocks == 1) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v[32];
                tmem_ld32(tA + lane_addr + 64 * half + 32 * c, v);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t to = bA + half * kSmallChunk + ns_sw(row, 4 * c + q);
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = ns_split_a(v[8 * q + 2 * e] * fa, v[8 * q + 2 * e + 1] * fa, l + e);
                    st_shared_v4(to, make_uint4(h[0], h[1], h[2], h[3]));
                    st_shared_v4(to + kSmallLo, make_uint4(l[0], l[1], l[2], l[3]));
                }
            }
        } else {
            // the row's columns of its diagonal block in fp32: rows of 512 bytes, their 16-byte pieces rotated
            // by the row against bank conflicts
            const bool any = kx > 0;   // a CTA past the last column adds nothing
            auto put = [&](int at, float v0, float v1, float v2, float v3) {
                st_shared_v4(bP + row * 512 + ((at ^ lane) << 4),
                             any ? make_uint4(__float_as_uint(v0), __float_as_uint(v1), __float_as_uint(v2), __float_as_uint(v3))
                                 : make_uint4(0, 0, 0, 0));
            };
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int cb = 64 * half + 32 * c;
                if (cb >> max(a.log_mp, 5) != quarter * 32 >> max(a.log_mp, 5)) continue;   // the same for the whole warp
                float v[32];
                tmem_ld32(tA + lane_addr + cb, v);
                if (mp >= 32) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) put((cb & (mp - 1)) / 4 + q, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                } else {   // blocks of 16: lanes 0-15 the first half, the others the second
                    const bool second = lane >= 16;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        put(q, second ? v[16 + 4 * q] : v[4 * q], second ? v[17 + 4 * q] : v[4 * q + 1],
                            second ? v[18 + 4 * q] : v[4 * q + 2], second ? v[19 + 4 * q] : v[4 * q + 3]);
                }
            }
            if (S > 1) cluster_sync();
            else __syncthreads();
            // Pieces of 16 bytes of the rows that this CTA adds: the thread's j-th is in row r0 + j * down, and its
            // terms come CTA by CTA and block by block, eight loads under way at a time, of as many pieces as they
            // belong to (16 x 128 x 512: 51 us, 300 x 64 x 2000: 422; one piece after the other they took 2.5 and 15 more; of eight
            // or more terms each the network between SMs is the limit, 100 x 4095, 68 us, took 1 less).
            const int log_pieces = a.log_mp - 2, log_blocks = 7 - a.log_mp, log_terms = a.log_ctas + log_blocks;
            const int at = threadIdx.x & ((1 << log_pieces) - 1), down = kSmallThreads >> log_pieces, terms = 1 << log_terms;
            const int r0 = (rank << (a.log_mp - a.log_ctas)) + ((int)threadIdx.x >> log_pieces);
            const int pieces = 1 << (a.log_mp - a.log_ctas + log_pieces);
            const int mine = (int)threadIdx.x < pieces ? max(1, pieces / kSmallThreads) : 0;
            const uint32_t lanes = pieces < 32 ? (1u << pieces) - 1 : 0xffffffffu;   // those with pieces, in the first warp
            auto exchange = [&](auto alone) {   // (with one CTA: plain shared memory)
                constexpr bool kAlone = decltype(alone)::value;
                auto give = [&](int j, const float4& sum) {
                    if (j >= mine) return;
                    // neighbouring lanes trade: the even one stores eight values of A, the odd one their rounding errors
                    uint32_t l0, l1;
                    const uint32_t h0 = ns_split_a(sum.x * fa, sum.y * fa, &l0), h1 = ns_split_a(sum.z * fa, sum.w * fa, &l1);
                    const bool odd = at & 1;
                    const uint32_t t0 = __shfl_xor_sync(lanes, odd ? h0 : l0, 1), t1 = __shfl_xor_sync(lanes, odd ? h1 : l1, 1);
                    const uint4 out = odd ? make_uint4(t0, t1, l0, l1) : make_uint4(h0, h1, t0, t1);
                    const int r = r0 + j * down;
                    for (int q = 0; q < blocks; ++q) {
                        const int col = (q << a.log_mp) + 4 * at;
                        const uint32_t to = (uint32_t)((col >> 6) * kSmallChunk) + ns_sw((q << a.log_mp) + r, (col & 63) >> 3) + (odd ? kSmallLo : 0);
                        if constexpr (kAlone) {
                            st_shared_v4(bA + to, out);
                        } else {
#pragma unroll 1
                            for (int b = 0; b < S; b += 2) {
                                st_cluster_v4(cluster_addr(sA, b) + to, out);
                                st_cluster_v4(cluster_addr(sA, b + 1) + to, out);
                            }
                        }
                    }
                };
                auto add = [](float4& sum, const float4& v) { sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w; };
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int u0 = 0; u0 >> log_terms < mine; u0 += 8) {
                    float4 v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {   // (past the thread's last piece: any of the buffer's, dropped)
                        const int t = (u0 + k) & (terms - 1);
                        const int br = (((t & (blocks - 1)) << a.log_mp) + r0 + ((u0 + k) >> log_terms) * down) & 127;
                        const uint32_t from = (uint32_t)(br * 512 + ((at ^ (br & 31)) << 4));
                        if constexpr (kAlone) {
                            const uint4 w = ld_shared_v4(bP + from);
                            v[k] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
                        } else {
                            v[k] = ld_cluster_f32x4(cluster_addr(sP, t >> log_blocks) + from);
                        }
                    }
                    if (terms == 2) {
#pragma unroll
                        for (int k = 0; k < 8; k += 2) {
                            add(v[k], v[k + 1]);
                            give((u0 + k) >> 1, v[k]);
                        }
                    } else if (terms == 4) {
#pragma unroll
                        for (int k = 0; k < 8; k += 4) {
#pragma unroll
                            for (int t = 1; t < 4; ++t) add(v[k], v[k + t]);
                            give((u0 + k) >> 2, v[k]);
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 8; ++t) add(sum, v[t]);
                        if (((u0 + 8) & (terms - 1)) == 0) {
                            give(u0 >> log_terms, sum);
                            sum = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                }
            };
            if (S == 1) exchange(std::true_type());
            else exchange(std::false_type());
            fence_proxy_async_all();
            if (S > 1) cluster_sync();   // A is whole in every CTA, and the partial sums have been read
        }
        fence_proxy_async_all();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (issues()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)   // A A, and A by twice its rounding error in the 128 columns that follow
                if (ks < km) {
                    const uint64_t d = sdesc_sw128(bA + (ks >> 2) * kSmallChunk + (ks & 3) * 32, 16, 1024);
                    mma_bf16(tX, d, d, kIdP, ks != 0);
                }
            commit();
        }
        wait_mma();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float v[32], w[32];
            tmem_ld32(tX + lane_addr + 64 * half + 32 * c, v);
            tmem_ld32(tX + lane_addr + 128 + 64 * half + 32 * c, w);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t to = half * kSmallChunk + ns_sw(row, 4 * c + q);
                const uint4 h = ld_shared_v4(bA + to), r = ld_shared_v4(bA + kSmallLo + to);
                const uint32_t wh[4] = {h.x, h.y, h.z, h.w}, wl[4] = {r.x, r.y, r.z, r.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float* b = v + 8 * q + 2 * e;
                    b[0] = fp * (b[0] + w[8 * q + 2 * e]);
                    b[1] = fp * (b[1] + w[8 * q + 2 * e + 1]);
                    fma_f16x2(b, wh[e], b_hi);
                    fma_f16x2(b, wh[e], b_lo);
                    fma_f16x2(b, wl[e], b_half);
                    hi[e] = ns_pack_half(b[0], b[1]);
                    fma_f16x2(b, hi[e], 0xbc00u);   // -1
                    lo[e] = ns_pack_half(b[0], b[1]);
                }
                st_shared_v4(bP + to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                st_shared_v4(bP + kSmallLo + to, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
        }
        fence_proxy_async_cta();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (issues()) {
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)   // B, then its rounding error, by X
                if ((ks & 7) < km)
                    mma_bf16(tX, sdesc_sw128(bP + ((ks & 7) >> 2) * kSmallChunk + (ks >> 3) * kSmallLo + (ks & 3) * 32, 16, 1024),
                             sdesc_sw128(bX + (ks & 7) * 2048, 16384, 1024), kIdX, ks != 0);
            commit();
        }
        wait_mma();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld32(tX + lane_addr + 128 * half + 32 * c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[32 * c + j] = fx * x[32 * c + j] + fv * v[j];
        }
        is = 1.f;
        if (s + 1 < a.steps) put_x(s + 2 == a.steps);
    }
    constexpr float u = 1.f / kXScale;
    if constexpr (VEC) {
        if (i < a.m) {
            __nv_bfloat16* o = a.O + ((long long)mat * a.m + i) * a.n + col0;
#pragma unroll
            for (int j = 0; j < 128; j += 8)
                if (col0 + j < a.n)
                    *reinterpret_cast<uint4*>(o + j) =
                        make_uint4(pack_bf16x2(x[j] * u, x[j + 1] * u), pack_bf16x2(x[j + 2] * u, x[j + 3] * u),
                                   pack_bf16x2(x[j + 4] * u, x[j + 5] * u), pack_bf16x2(x[j + 6] * u, x[j + 7] * u));
        }
    } else {
        constexpr int kPitch = kSmallCols * 2 + 4;
        const uint32_t stage = smem_u32(smem);
        const NsSlab slab{a.m, a.n, a.log_mp, a.flip, rank * blocks * kSmallCols};
        __nv_bfloat16* o = a.O + (long long)mat * a.m * a.n;
        const uint32_t past = (uint32_t)reinterpret_cast<uintptr_t>(o + (a.flip ? slab.cta0 * a.m : i * a.n + slab.cta0));
        const uint32_t to = a.flip ? stage + (past & 15) + (uint32_t)(((block * kSmallCols + half * 128) * a.m + i) * 2)
                                   : stage + (past & 3) + (uint32_t)(row * kPitch + half * 256);
        const uint32_t step = a.flip ? a.m * 2 : 2;
#pragma unroll
        for (int j = 0; j < 128; ++j)
            asm volatile("{\n.reg .pred p;\nsetp.lt.s32 p, %2, %3;\n@p st.shared.b16 [%0], %1;\n}" ::"r"(to + j * step),
                         "h"(__bfloat16_as_ushort(__float2bfloat16_rn(x[j] * u))), "r"(j), "r"(left) : "memory");
        __syncthreads();
        slab.each(kPitch, warp, [&](const NsRun& run) {
            if (a.flip) ns_stage_out<16, kSmallThreads>(o + run.first, stage, 2 * run.count);
            else ns_stage_out<4, 32>(o + run.first, stage + run.at, 2 * run.count);
        });
    }
    // an MMA whose wait ran out may still be at work (bounded): it ends before its memory is given up
    if (*abort_flag && threadIdx.x == 0 && *open >= 0) ns_wait_drain(done, (uint32_t)*open);
    tc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();   // no CTA's shared memory is read or written any more
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- launches --------------------------------------------------------------------------------------
static int ns_log2(int v) { return v < 2 ? 0 : 1 + ns_log2(v / 2); }

struct NsLayout {
    int64_t N, m, n, lda, ldx, parts;
    bool ab_lo;
    size_t partial, inv_s, done, A, B, x0, x1, lo, total;
};

static bool ns_layout(int64_t N, int64_t R, int64_t C, NsLayout* L) {
    if (N < 0 || R < 1 || C < 1) return false;
    L->N = N;
    L->m = std::min(R, C);
    L->n = std::max(R, C);
    L->lda = (L->m + 7) / 8 * 8;   // rows on 16-byte boundaries for the TMA
    L->ldx = (L->n + 7) / 8 * 8;
    L->parts = std::min<int64_t>(kNormParts, (R * C + kNormPart - 1) / kNormPart);
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
    take(256);   // status word
    if (L->m <= kTinyRows) {
        L->total = o;
        return true;
    }
    int mp;
    const int S = ns_small_cluster(N, L->m, L->n, &mp);
    if (S > 0 && S <= 8) {   // (whether a cluster of 16 is possible only the GPU can tell)
        L->total = o;
        return true;
    }
    L->partial = take((size_t)N * L->parts * 4);
    L->inv_s = take((size_t)N * 4);
    L->done = take((size_t)N * (1 + 2 * ((L->m + 127) / 128)) * 4);   // counters (tile rows of 128, or fewer of 256)
    L->ab_lo = L->m <= 128;
    L->A = take((size_t)N * (L->ab_lo ? 2 : 1) * L->m * L->lda * 2);
    L->B = take((size_t)N * (L->ab_lo ? 2 : 1) * L->m * L->lda * 2);
    L->x0 = take((size_t)N * L->m * L->ldx * 2);
    L->x1 = take((size_t)N * L->m * L->ldx * 2);
    L->lo = take((size_t)N * L->m * L->ldx * 2);
    L->total = o;
    return true;
}

size_t orthogonalise_workspace(int64_t N, int64_t R, int64_t C) {
    NsLayout L;
    return ns_layout(N, R, C, &L) ? L.total : 0;
}

// The most CTAs that are resident at once, and the launch of that many (or one, or a pair, for each unit):
// cooperative, since CTAs wait for one another's tiles.
template <bool PAIR>
static cudaError_t ns_steps(cudaStream_t st, int most, const NsMaps& maps, const NsArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = PAIR ? 2 : 1;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(PAIR ? 2 * std::min(a.units, most / 2) : std::min(a.units, most));
    cfg.blockDim = dim3(kNsThreads);
    cfg.dynamicSmemBytes = kNsSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ns_steps_kernel<PAIR>, maps, a);
}
template <bool PAIR>
static cudaError_t ns_resident(int device, int num_sms, int* most) {
    static PerDevice<int> held;
    return held.get(device, most, [&](int* ctas) {
        auto kern = ns_steps_kernel<PAIR>;
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem);
        *ctas = num_sms;
        if (err == cudaSuccess && PAIR) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 2;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(num_sms / 2 * 2);
            cfg.blockDim = dim3(kNsThreads);
            cfg.dynamicSmemBytes = kNsSmem;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int clusters = 0;
            err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
            *ctas = 2 * std::max(1, std::min(clusters, num_sms / 2));
        }
        return err;
    });
}

template <typename T>
static cudaError_t ns_tiny(cudaStream_t st, const T* G, __nv_bfloat16* O, const NsLayout& L, bool flip, int steps,
                           const float* coeffs, float eps) {
    int S = 1;
    while (S < 8 && S * 2 * kTinyThreads < L.n) S *= 2;
    NsTiny a{(int)L.m, (int)L.n, flip, steps, S, eps};
    std::copy(coeffs, coeffs + 3 * steps, a.co);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(L.N * S));
    cfg.blockDim = dim3(kTinyThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ns_tiny_kernel<T>, G, O, a);
}

// `*ran` false: this GPU has no room for such a cluster
template <typename T, bool VEC>
static cudaError_t ns_small(cudaStream_t st, int device, const T* G, int S, int N, const NsSmall& a, bool* ran) {
    auto kern = ns_small_kernel<T, VEC>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = S;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(S, N);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = kSmallBytes;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    static PerDevice<bool> held;
    bool sixteen = false;
    const cudaError_t err = held.get(device, &sixteen, [&](bool* fits) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallBytes);
        if (e != cudaSuccess) return e;
        *fits = false;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
            cudaLaunchConfig_t c16 = cfg;
            cudaLaunchAttribute a16 = at[0];
            a16.val.clusterDim.x = 16;
            c16.gridDim = dim3(16, 1);
            c16.attrs = &a16;
            c16.numAttrs = 1;
            int clusters = 0;
            *fits = cudaOccupancyMaxActiveClusters(&clusters, kern, &c16) == cudaSuccess && clusters > 0;
        }
        if (!*fits) cudaGetLastError();   // an answer, not an error of this call
        return cudaSuccess;
    });
    if (err != cudaSuccess) return err;
    *ran = S <= 8 || sixteen;
    return *ran ? cudaLaunchKernelEx(&cfg, kern, G, a) : cudaSuccess;
}

template <typename T>
static cudaError_t ns_first_x(cudaStream_t st, const NsLayout& L, const T* G, int R, int C, float eps, char* w, bool lo,
                              int counts, int num_sms) {
    float* partial = reinterpret_cast<float*>(w + L.partial);
    const long long elems = (long long)R * C;
    const unsigned N = (unsigned)L.N;
    const dim3 parts((unsigned)L.parts, N);
    cudaError_t err = launch_pdl(ns_norm_kernel<T>, parts, 256, 0, st, G, elems, (int)L.parts, partial);
    if (err != cudaSuccess) return err;
    const NsPrep p{partial, reinterpret_cast<__half*>(w + L.x0), lo ? reinterpret_cast<__half*>(w + L.lo) : nullptr,
                   reinterpret_cast<float*>(w + L.inv_s), reinterpret_cast<int*>(w + L.done), counts, (int)L.parts, R, C, (int)L.ldx, eps, R > C};
    const auto blocks = [](int64_t items, int64_t per) { return (unsigned)((items + per - 1) / per); };
    if (R > C) {
        // one tile a block until there are several for each block that an SM holds
        const int per = (int64_t)N * blocks(C, 64) * blocks(R, 64) > 16 * num_sms ? 4 : 1;
        const dim3 grid(blocks(C, 64), blocks(R, 64 * per), N);
        return C % 8 != 0 ? launch_pdl(ns_prep_flip_kernel<T, false>, grid, 256, 0, st, G, p, per)
                          : launch_pdl(ns_prep_flip_kernel<T, true>, grid, 256, 0, st, G, p, per);
    }
    if (C % 8 != 0) return launch_pdl(ns_prep_rows_kernel<T>, dim3(blocks(R * L.ldx, 8 * 256), N), 256, 0, st, G, p);
    return launch_pdl(ns_prep_kernel<T>, dim3(blocks(elems, 8 * 256 * kPrepPer), N), 256, 0, st, G, p);
}

cudaError_t launch_orthogonalise(cudaStream_t st, const void* G, bool g_f32, int64_t N, int64_t R, int64_t C, void* O,
                                 int steps, const float* coeffs, float eps, void* workspace, int num_sms, int* status,
                                 long long wait_limit, bool withhold_loads) {
    NsLayout L;
    if (!ns_layout(N, R, C, &L)) return cudaErrorInvalidValue;
    if (L.m <= kTinyRows) {
        return g_f32 ? ns_tiny(st, static_cast<const float*>(G), static_cast<__nv_bfloat16*>(O), L, R > C, steps, coeffs, eps)
                     : ns_tiny(st, static_cast<const __nv_bfloat16*>(G), static_cast<__nv_bfloat16*>(O), L, R > C, steps, coeffs, eps);
    }
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess) return err;
    int mp;
    if (const int S = ns_small_cluster(N, L.m, L.n, &mp)) {
        NsSmall a{(int)R, (int)C, (int)L.m, (int)L.n, mp, ns_log2(mp), ns_log2(S), steps, R > C, eps};
        std::copy(coeffs, coeffs + 3 * steps, a.co);
        a.O = static_cast<__nv_bfloat16*>(O);
        a.status = status;
        a.wait_limit = wait_limit > 0 ? wait_limit : kWaitTimeoutCycles;
        a.withhold = withhold_loads;
        const auto* gf = static_cast<const float*>(G);
        const auto* gb = static_cast<const __nv_bfloat16*>(G);
        bool ran = false;
        err = C % 8 == 0 && R <= C ? (g_f32 ? ns_small<float, true>(st, device, gf, S, (int)N, a, &ran)
                                                    : ns_small<__nv_bfloat16, true>(st, device, gb, S, (int)N, a, &ran))
                                           : (g_f32 ? ns_small<float, false>(st, device, gf, S, (int)N, a, &ran)
                                                    : ns_small<__nv_bfloat16, false>(st, device, gb, S, (int)N, a, &ran));
        if (err != cudaSuccess || ran) return err;
    }
    char* w = static_cast<char*>(workspace);
    const bool flip = R > C;
    const int64_t m = L.m, n = L.n;
    // Pairs take in half as much for the same product, but a tile of theirs is four of one CTA's, and few of them leave
    // SMs idle.  Even at about half a tile of X for each SM, sooner for a few large matrices, later for several small
    // ones (us by pairs and by single CTAs; tiles of a pair in X): 1 x 2048 x 2048 (64) 253 and 274, 76 x 200 x 200 (76) 123
    // and 131, 150 x 200 x 200 (150) 179 and 245, 40 x 300 x 400 (160) 158 and 168, 6 x 1024 x 1024 (96) 209 and 213;
    // 3 x 777 x 1001 (48) 195 and 157, 5 x 777 x 1001 (80) 194 and 180, 9 x 600 x 600 (81) 188 and 168.
    const bool pair = m > 128 && N * ((m + 255) / 256) * ((n + 255) / 256) >= num_sms / 2;
    const int tile = pair ? 256 : 128;
    const int mt = (int)((m + tile - 1) / tile), nt = (int)((n + tile - 1) / tile);
    err =
        g_f32 ? ns_first_x(st, L, static_cast<const float*>(G), (int)R, (int)C, eps, w, steps > 1, 1 + 2 * mt, num_sms)
              : ns_first_x(st, L, static_cast<const __nv_bfloat16*>(G), (int)R, (int)C, eps, w, false, 1 + 2 * mt, num_sms);
    if (err != cudaSuccess) return err;
    NsMaps t;
    auto map = [&](CUtensorMap* out, size_t at, int64_t cols, int64_t ld, int64_t batch, int rows) {
        return tmap_batched(out, w + at, false, cols, m, ld, batch, rows);
    };
    const int64_t nab = L.ab_lo ? 2 * N : N;
    bool ok = map(&t.a, L.A, m, L.lda, nab, 128) && map(&t.a_t, L.A, m, L.lda, N, 64) &&
              map(&t.b, L.B, m, L.lda, nab, 128) && map(&t.b_t, L.B, m, L.lda, N, 64) &&
              map(&t.x[0], L.x0, n, L.ldx, N, 128) && map(&t.x[1], L.x1, n, L.ldx, N, 128) &&
              map(&t.x_t[0], L.x0, n, L.ldx, N, 64) && map(&t.x_t[1], L.x1, n, L.ldx, N, 64) &&
              map(&t.lo, L.lo, n, L.ldx, N, 128);
    const bool o_box = C % 8 == 0;   // O's rows are multiples of 16 bytes
    t.o = t.o_t = t.a;
    if (o_box) ok = ok && tmap_batched(&t.o, O, true, C, R, C, N, 128) && tmap_batched(&t.o_t, O, true, C, R, C, N, 64);
    if (!ok) return cudaErrorInvalidValue;
    int most = 0;
    if ((err = pair ? ns_resident<true>(device, num_sms, &most) : ns_resident<false>(device, num_sms, &most)) != cudaSuccess) return err;
    const int ctas = pair ? most / 2 : most;
    NsArgs a{};
    a.m = (int)m; a.n = (int)n; a.N = (int)N;
    a.steps = steps;
    a.mt = mt; a.nt = nt;
    a.tri = a.mt * (a.mt + 1) / 2; a.full = a.mt * a.nt;
    a.parts = pair ? 2 : 1;
    a.last_parts = pair && m - (int64_t)(mt - 1) * tile <= 128 ? 1 : a.parts;
    // a wave and a quarter of triangle tiles in a half group, the groups equal: fewer and a phase waits for
    // the last tiles of the one before, more and X leaves L2 in between (256 x 768 x 2048: 6.8, 6.2, 6.1, 6.2
    // and 6.3 ms with 6, 9, 12, 20 and 64 matrices in a half)
    const int64_t most_h = std::max<int64_t>(1, (5 * ctas + 4 * a.tri - 1) / (4 * a.tri));
    a.supers = (int)((N + 2 * most_h - 1) / (2 * most_h));
    a.halves = N > 1 ? 2 : 1;
    a.h = (int)((N + a.halves * a.supers - 1) / (a.halves * a.supers));
    a.supers = ((int)N + a.halves * a.h - 1) / (a.halves * a.h);
    a.per_cycle = a.halves * a.h * (2 * a.tri + a.full);
    a.cycles = a.supers * steps + (a.halves - 1);
    if ((int64_t)a.cycles * a.per_cycle >= INT32_MAX) return cudaErrorInvalidValue;
    a.units = a.cycles * a.per_cycle;
    a.k_gram = (int)((n + 63) / 64); a.k_poly = (int)((m + 63) / 64);
    a.ab_lo = L.ab_lo;
    a.first_lo = g_f32;
    a.out_kind = o_box ? (flip ? NS_O_BOX_FLIP : NS_O_BOX) : (flip ? NS_O_PLAIN_FLIP : NS_O_PLAIN);
    std::copy(coeffs, coeffs + 3 * steps, a.co);
    a.inv_s = reinterpret_cast<float*>(w + L.inv_s);
    a.done = reinterpret_cast<int*>(w + L.done);
    a.O = static_cast<__nv_bfloat16*>(O);
    a.status = status;
    a.wait_limit = wait_limit > 0 ? wait_limit : kWaitTimeoutCycles;
    a.withhold_loads = withhold_loads;
    return pair ? ns_steps<true>(st, most, t, a) : ns_steps<false>(st, most, t, a);
}

}  // namespace moe
