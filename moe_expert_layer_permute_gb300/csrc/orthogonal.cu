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
// 0.1 %.  A matrix of up to 128 rows keeps B's rounding error too, as a second product of APPLY: with few
// singular values B's error does not average out (a single row came out up to 0.5 % off).
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace moe {

constexpr float kXScale = 256.f, kABScale = 1024.f, kLoScale = 2048.f;
constexpr int kNsStages = 4;
constexpr int kNsEpi = 8;          // epilogue warps: two for each quarter of the TMEM lanes, on alternate columns
constexpr int kNsThreads = 64 + 32 * kNsEpi;
constexpr int kNsSlots = 3;        // pairs of boxes per epilogue warp
constexpr int kNsBox = 2048;       // a box: 32 rows x 32 16-bit values
constexpr int kNsSmem = 1024 + kNsStages * 32768 + kNsEpi * kNsSlots * 2 * kNsBox + 512;
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

// Part blockIdx.x of matrix blockIdx.y's sum of squares; VEC: the matrices are multiples of 8 elements.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) ns_norm_kernel(const T* G, long long elems, int parts, float* partial) {
    grid_dep_wait();
    const T* g = G + (long long)blockIdx.y * elems;
    float v = 0.f;
    if constexpr (VEC) {
#pragma unroll 4
        for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < elems; i += (long long)parts * 2048) {
            float x[8];
            ns_val8(x, g + i);
            float s = x[0] * x[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) s += x[j] * x[j];
            v += s;
        }
    } else {
        for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < elems; i += (long long)parts * 256) {
            const float x = ns_val(g, i);
            v += x * x;
        }
    }
    v = ns_block_sum(v);
    if (threadIdx.x == 0) partial[(long long)blockIdx.y * parts + blockIdx.x] = v;
}

// The power of two p with |G| p in [1/2, 1) (1 for |G| = 0), and inv_s = 1 / ((|G| + eps) p), so that the
// first X is G p inv_s.  A norm that is not finite makes the whole matrix NaN.
__device__ __forceinline__ float ns_split(float norm, float eps, float* inv_s) {
    const int ex = (int)((__float_as_uint(norm) >> 23) & 0xffu) - 126;   // -62 .. 64: a root of an fp32 sum
    const bool fine = norm <= 3.4e38f;
    const float p = norm < 1e-30f ? 1.f : __uint_as_float((uint32_t)(127 - ex) << 23);
    *inv_s = fine ? 1.f / ((norm + eps) * p) : NAN;
    return fine ? p : NAN;
}

struct NsPrep {
    const float* partial;
    __half* hi;
    __half* lo;      // null where G is exact in fp16 (bf16 G)
    float* inv_s;    // [N]
    int parts, R, C, ld;
    float eps;
    int flip;        // store G^T
};

// The factor of matrix `mat`'s first X from its partial sums; `first` also records inv_s.
__device__ __forceinline__ float ns_factor(const NsPrep& a, int mat, bool first) {
    float v = 0.f;
    for (int i = threadIdx.x; i < a.parts; i += 256) v += a.partial[(long long)mat * a.parts + i];
    float inv_s;
    const float f = ns_split(sqrtf(ns_block_sum(v)), a.eps, &inv_s) * kXScale;
    if (first && threadIdx.x == 0) a.inv_s[mat] = inv_s;
    return f;
}
__device__ __forceinline__ uint32_t ns_pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 ns_unpack_half(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
// eight values of X, and their rounding errors, at a 16-byte boundary
__device__ __forceinline__ void ns_store8(const NsPrep& a, long long at, const float* x) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = ns_pack_half(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<uint4*>(a.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    if (!a.lo) return;
    uint32_t l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = ns_unpack_half(h[j]);
        l[j] = ns_pack_half((x[2 * j] - f.x) * kLoScale, (x[2 * j + 1] - f.y) * kLoScale);
    }
    *reinterpret_cast<uint4*>(a.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

// Rows of multiples of 8 elements, as they stand: X's pitch is C and the matrix one run of elements.
constexpr int kPrepPer = 4;   // runs of eight per thread
template <typename T>
__global__ void __launch_bounds__(256) ns_prep_kernel(const T* G, const NsPrep a) {
    grid_dep_wait();
    const int mat = blockIdx.y;
    const long long elems = (long long)a.R * a.C;
    const float f = ns_factor(a, mat, blockIdx.x == 0);
#pragma unroll
    for (int q = 0; q < kPrepPer; ++q) {
        const long long i = (((long long)blockIdx.x * kPrepPer + q) * 256 + threadIdx.x) * 8;
        if (i >= elems) break;
        float x[8];
        ns_val8(x, G + mat * elems + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= f;
        ns_store8(a, mat * elems + i, x);
    }
}

// G^T for rows of multiples of 8 elements: 64 x 64 tiles through shared memory, 16 bytes a load and 32 a
// store (the pitch is a multiple of 16 bytes; what is past R in a row's last 16 is never read).
template <typename T>
__global__ void __launch_bounds__(256) ns_prep_flip_kernel(const T* G, const NsPrep a) {
    grid_dep_wait();
    __shared__ float tile[64][65];
    const int mat = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    const float f = ns_factor(a, mat, blockIdx.x == 0 && blockIdx.y == 0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = q * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
        if (r0 + r < a.R && c0 + c < a.C) ns_val8(x, G + ((long long)mat * a.R + r0 + r) * a.C + c0 + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[r][c + j] = x[j] * f;
    }
    __syncthreads();
    const int c = threadIdx.x & 63, r = (threadIdx.x >> 6) * 16;
    if (c0 + c >= a.C) return;
#pragma unroll
    for (int q = 0; q < 16; q += 8) {
        if (r0 + r + q >= a.R) break;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = tile[r + q + j][c];
        ns_store8(a, ((long long)mat * a.C + c0 + c) * a.ld + r0 + r + q, x);
    }
}

// Any size: 32 x 32 tiles, an element at a time.
template <typename T>
__global__ void __launch_bounds__(256) ns_prep_any_kernel(const T* G, const NsPrep a) {
    grid_dep_wait();
    __shared__ float tile[32][33];
    const int mat = blockIdx.z, r0 = blockIdx.y * 32, c0 = blockIdx.x * 32;
    const float f = ns_factor(a, mat, blockIdx.x == 0 && blockIdx.y == 0);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int rows = a.flip ? a.C : a.R, cols = a.flip ? a.R : a.C;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        const int r = r0 + ty + j, c = c0 + tx;
        tile[ty + j][tx] = r < a.R && c < a.C ? ns_val(G, ((long long)mat * a.R + r) * a.C + c) * f : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        const int r = (a.flip ? c0 : r0) + ty + j, c = (a.flip ? r0 : c0) + tx;
        if (r >= rows || c >= cols) continue;
        const float x = a.flip ? tile[tx][ty + j] : tile[ty + j][tx];
        const __half h = __float2half_rn(x);
        const long long at = ((long long)mat * rows + r) * a.ld + c;
        a.hi[at] = h;
        if (a.lo) a.lo[at] = __float2half_rn((x - __half2float(h)) * kLoScale);
    }
}

// ---- the three products ------------------------------------------------------------------------------
enum NsMode { NS_GRAM = 0, NS_POLY, NS_APPLY };
// How the last step stores O: not at all (an inner step), through TMA boxes as it stands or flipped, or
// by plain stores where its rows are not multiples of 16 bytes
enum NsOut { NS_O_NONE = 0, NS_O_BOX, NS_O_BOX_FLIP, NS_O_PLAIN, NS_O_PLAIN_FLIP };

struct NsArgs {
    int m, n, lda, ldx;
    int tiles_n, tiles;          // tile columns (APPLY), tiles per matrix
    int units;                   // tiles of the whole batch
    int k_blocks;
    int k_wrap;                  // k_blocks, or half of them: APPLY with B's rounding error as a second B
    int batch;                   // N: matrix N + i of the B array is the rounding error of matrix i's B
    float a, b, c;
    const float* inv_s;          // [N] in the first step, null after it
    int xlo;                     // APPLY: X has a rounding error (else it is exact, or the step takes none)
    int keep_lo;                 // POLY: store B's rounding error; APPLY: the next X's
    int out_kind;                // NsOut
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

struct NsTile {
    int mat, i, j;
};
template <int MODE>
__device__ __forceinline__ NsTile ns_tile(int unit, const NsArgs& a) {
    NsTile t;
    t.mat = unit / a.tiles;
    int left = unit - t.mat * a.tiles;
    if (MODE == NS_APPLY) {
        t.i = left / a.tiles_n;
        t.j = left - t.i * a.tiles_n;
    } else {
        t.i = 0;
        while (left > t.i) left -= ++t.i;   // row i of the lower triangle has i + 1 tiles
        t.j = left;
    }
    return t;
}

// A warp's output boxes: 32 rows x 64 bytes (32 16-bit values), 64-byte swizzle.
// the lane's row of 32 values, packed in pairs
__device__ __forceinline__ void ns_box_row(uint32_t box, int lane, const uint32_t* v) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        st_shared_v4(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
}
// the transpose: the lane's value j goes to row j, column lane
__device__ __forceinline__ void ns_box_col(uint32_t box, int lane, const uint32_t* v) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint16_t h = (uint16_t)(j & 1 ? v[j >> 1] >> 16 : v[j >> 1] & 0xffffu);
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(box + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) + (lane & 7) * 2), "h"(h)
                     : "memory");
    }
}
__device__ __forceinline__ void ns_box_read(uint32_t* v, uint32_t box, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 w = ld_shared_v4(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4));
        v[4 * q] = w.x; v[4 * q + 1] = w.y; v[4 * q + 2] = w.z; v[4 * q + 3] = w.w;
    }
}

// The chunks of 32 columns that an epilogue warp works through (every second one), tile after tile.
template <int MODE, int TILE>
struct NsChunks {
    int u, stride, rank, quarter, half;
    NsTile t;
    int row0, n0, c, cols;   // the warp's first row, the tile's first column, the chunk, the columns to cover
    __device__ __forceinline__ void tile(const NsArgs& a) {
        t = ns_tile<MODE>(u, a);
        row0 = t.i * TILE + rank * 128 + quarter * 32;
        n0 = t.j * TILE;
        c = 32 * half;
        cols = row0 < a.m ? min(TILE, (MODE == NS_APPLY ? a.n : a.m) - n0) : 0;
    }
    // moves over tiles without a chunk for this warp; false past the last unit
    __device__ __forceinline__ bool settle(const NsArgs& a) {
        while (u < a.units && c >= cols) {
            u += stride;
            if (u < a.units) tile(a);
        }
        return u < a.units;
    }
};

// Persistent blocks walk the batch's tiles.  Warp 0 loads, warp 1 issues the MMAs, eight warps store (see
// gemm.cu for the scheme): four stages of 32 KB, two accumulators, waits bounded.  What an epilogue needs
// besides its accumulator (POLY: A; APPLY: X and its rounding error) comes by TMA into the warp's ring of
// three slots, two chunks of 32 columns ahead and across tiles: with loads into registers a chunk ahead
// APPLY waited on memory (256 x 768 x 2048: 851 us a launch).  The results replace it in place and leave
// by TMA from there.
//   PAIR: two CTAs share a 256 x 256 tile (cta_group::2), each holding 128 rows of the first operand and
//   half of the second; otherwise one CTA computes 128 x 128.
// GRAM and POLY are symmetric: tiles of the lower triangle alone, and those below the diagonal are stored
// twice, as they are and transposed through shared memory.  Operands: GRAM rows of X by rows of X, POLY
// rows of A by rows of A (A = A^T), both contiguous along K; APPLY rows of B by columns of X (contiguous
// along N).  The TMA fills K past the edge with zeros and drops stores outside a matrix, so no size needs
// padding beyond 16-byte rows.
template <int MODE, bool PAIR>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmL,
                   const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD, const NsArgs a) {
    grid_dep_wait();
    constexpr int kTile = PAIR ? 256 : 128;      // rows and columns of a unit's tile
    constexpr int kOperand = 128 * 128;          // bytes of one operand's K slice per CTA: 128 x 64 fp16
    constexpr bool kBmn = MODE == NS_APPLY;
    constexpr uint32_t kIdesc = idesc_f16(kTile, kTile, false, kBmn);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + kNsStages * kOperand;
    uint8_t* sBox = sB + kNsStages * kOperand;
    uint64_t* full = reinterpret_cast<uint64_t*>(sBox + kNsEpi * kNsSlots * 2 * kNsBox);
    uint64_t* empty = full + kNsStages;
    uint64_t* tfull = empty + kNsStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* slot_full = drain + 1;             // [kNsEpi][kNsSlots]
    uint32_t* tslot = reinterpret_cast<uint32_t*>(slot_full + kNsEpi * kNsSlots);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
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
        for (int i = 0; i < kNsEpi * kNsSlots; ++i) mbar_init(slot_full + i, 1);
        *abort_flag = 0;
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

    if (warp == 0) {
        if (lane == 0 && !a.withhold_loads) {
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int u = unit0; u < a.units && ok; u += stride) {
                const NsTile t = ns_tile<MODE>(u, a);
                const int m0 = t.i * kTile + rank * 128, n0 = t.j * kTile + rank * 128;
                for (int kb = 0; kb < a.k_blocks; ++kb) {
                    if (!mbar_wait(empty + stage, phase ^ 1u, abort_flag, a.status, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    uint8_t* dA = sA + stage * kOperand;
                    uint8_t* dB = sB + stage * kOperand;
                    const bool second = kb >= a.k_wrap;
                    const int k0 = (second ? kb - a.k_wrap : kb) * 64;
                    const int matA = second ? t.mat + a.batch : t.mat;
                    if constexpr (PAIR) {
                        // both CTAs' copies land on the leader's barrier, which expects both
                        const uint32_t lbar = cluster_addr(full + stage, 0);
                        if (rank == 0) mbar_arrive_expect_tx(full + stage, 4 * kOperand);
                        tma_load_3d_pair(dA, &tmA, lbar, k0, m0, matA);
                        if (kBmn) {
                            tma_load_3d_pair(dB, &tmB, lbar, n0, k0, t.mat);
                            tma_load_3d_pair(dB + kOperand / 2, &tmB, lbar, n0 + 64, k0, t.mat);
                        } else {
                            tma_load_3d_pair(dB, &tmB, lbar, k0, n0, t.mat);
                        }
                    } else {
                        mbar_arrive_expect_tx(full + stage, 2 * kOperand);
                        tma_load_3d(dA, &tmA, full + stage, k0, m0, matA);
                        if (kBmn) {
                            tma_load_3d(dB, &tmB, full + stage, n0, k0, t.mat);
                            tma_load_3d(dB + kOperand / 2, &tmB, full + stage, n0 + 64, k0, t.mat);
                        } else {
                            tma_load_3d(dB, &tmB, full + stage, k0, n0, t.mat);
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
            for (int u = unit0; u < a.units && ok; u += stride) {
                if (!(PAIR ? mbar_wait_cluster(tempty + acc, acc_phase ^ 1u, abort_flag, a.status, a.wait_limit)
                           : mbar_wait(tempty + acc, acc_phase ^ 1u, abort_flag, a.status, a.wait_limit))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * kTile);
                for (int kb = 0; kb < a.k_blocks; ++kb) {
                    if (!mbar_wait(full + stage, phase, abort_flag, a.status, a.wait_limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = a_base + stage * kOperand, sb = b_base + stage * kOperand;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = sdesc_sw128(sa + ks * 32, 16, 1024);
                        const uint64_t bd = kBmn ? sdesc_sw128(sb + ks * 2048, kOperand / 2, 1024)
                                                 : sdesc_sw128(sb + ks * 32, 16, 1024);
                        if constexpr (PAIR) mma_bf16_pair(d, ad, bd, kIdesc, (kb | ks) != 0);
                        else mma_bf16(d, ad, bd, kIdesc, (kb | ks) != 0);
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
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        uint8_t* boxes = sBox + (warp - 2) * kNsSlots * 2 * kNsBox;
        uint64_t* box_full = slot_full + (warp - 2) * kNsSlots;
        constexpr bool kLoads = MODE != NS_GRAM;
        const bool two = MODE == NS_APPLY && a.xlo;
        using Chunks = NsChunks<MODE, kTile>;
        Chunks cur{unit0, stride, rank, quarter, half}, ahead{unit0, stride, rank, quarter, half};
        if (unit0 < a.units) {
            cur.tile(a);
            ahead.tile(a);
        }
        uint32_t loaded = 0, used = 0;   // chunks requested and worked on; slot: mod kNsSlots
        auto request = [&] {             // the next chunk's boxes (lane 0)
            if (!ahead.settle(a)) return;
            uint64_t* bar = box_full + loaded % kNsSlots;
            uint8_t* dst = boxes + (loaded % kNsSlots) * 2 * kNsBox;
            mbar_arrive_expect_tx(bar, two ? 2 * kNsBox : kNsBox);
            tma_load_3d(dst, &tmX, bar, ahead.n0 + ahead.c, ahead.row0, ahead.t.mat);
            if (two) tma_load_3d(dst + kNsBox, &tmL, bar, ahead.n0 + ahead.c, ahead.row0, ahead.t.mat);
            ahead.c += 64;
            ++loaded;
        };
        if (kLoads && lane == 0 && !a.withhold_loads)
            for (int i = 0; i < kNsSlots - 1; ++i) request();
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (; cur.u < a.units && ok; cur.u += stride) {
            cur.tile(a);
            const NsTile t = cur.t;
            const int row0 = cur.row0, r = row0 + lane;
            const float is = a.inv_s ? __ldg(a.inv_s + t.mat) : 1.f;
            if (!__all_sync(0xffffffffu, mbar_wait(tfull + acc, acc_phase, abort_flag, a.status, a.wait_limit))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 32 * half; c0 < cur.cols; c0 += 64, ++used) {
                const int col = cur.n0 + c0;
                uint8_t* box = boxes + (used % kNsSlots) * 2 * kNsBox;
                const uint32_t sbox = smem_u32(box);
                float v[32];
                uint32_t out[16], low[16];
                tmem_ld32(tmem + lane_addr + (uint32_t)(acc * kTile + c0), v);
                if (kLoads) {
                    ok = __all_sync(0xffffffffu, mbar_wait(box_full + used % kNsSlots, used / kNsSlots & 1, abort_flag,
                                                           a.status, a.wait_limit));
                    if (!ok) break;
                } else {
                    if (lane == 0) bulk_wait_read<kNsSlots - 1>();   // the slot's last store has read it
                    __syncwarp();
                }
                if constexpr (MODE == NS_GRAM) {
                    const float f = kABScale / (kXScale * kXScale) * is * is;
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = ns_pack_half(v[2 * j] * f, v[2 * j + 1] * f);
                } else if constexpr (MODE == NS_POLY) {
                    ns_box_read(out, sbox, lane);
                    const float fc = a.c / kABScale;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = ns_unpack_half(out[j]);
                        v[2 * j] = a.b * x.x + fc * v[2 * j];
                        v[2 * j + 1] = a.b * x.y + fc * v[2 * j + 1];
                        out[j] = ns_pack_half(v[2 * j], v[2 * j + 1]);
                    }
                    if (a.keep_lo) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 h = ns_unpack_half(out[j]);
                            low[j] = ns_pack_half(v[2 * j] - h.x, v[2 * j + 1] - h.y);
                        }
                    }
                } else {
                    ns_box_read(out, sbox, lane);
                    const float fd = is * (1.f / kABScale), fx = is * a.a;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = ns_unpack_half(out[j]);
                        v[2 * j] = fx * x.x + fd * v[2 * j];
                        v[2 * j + 1] = fx * x.y + fd * v[2 * j + 1];
                    }
                    if (two) {
                        ns_box_read(low, sbox + kNsBox, lane);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 x = ns_unpack_half(low[j]);
                            v[2 * j] += fx * (1.f / kLoScale) * x.x;
                            v[2 * j + 1] += fx * (1.f / kLoScale) * x.y;
                        }
                    }
                    if (a.out_kind == NS_O_NONE) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) out[j] = ns_pack_half(v[2 * j], v[2 * j + 1]);
                        if (a.keep_lo) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 h = ns_unpack_half(out[j]);
                                low[j] = ns_pack_half((v[2 * j] - h.x) * kLoScale, (v[2 * j + 1] - h.y) * kLoScale);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            out[j] = pack_bf16x2(v[2 * j] * (1.f / kXScale), v[2 * j + 1] * (1.f / kXScale));
                    }
                }
                const bool flip = MODE == NS_APPLY && a.out_kind == NS_O_BOX_FLIP;
                const bool plain = MODE == NS_APPLY && a.out_kind == NS_O_PLAIN;
                const bool plain_flip = MODE == NS_APPLY && a.out_kind == NS_O_PLAIN_FLIP;
                // the second box: the transpose of a tile below the diagonal, or the rounding error
                const bool twin = MODE != NS_APPLY && t.i != t.j;
                const bool with_lo = MODE != NS_GRAM && a.keep_lo;
                __syncwarp();   // every lane has read the boxes
                if (plain_flip) {   // a warp's 32 rows are 64 consecutive bytes of O
                    if (r < a.m) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < a.n)
                                reinterpret_cast<uint16_t*>(a.O)[((long long)t.mat * a.n + col + j) * a.m + r] =
                                    (uint16_t)(j & 1 ? out[j >> 1] >> 16 : out[j >> 1]);
                    }
                } else {
                    if (flip) ns_box_col(sbox, lane, out);
                    else ns_box_row(sbox, lane, out);
                    if (twin) ns_box_col(sbox + kNsBox, lane, out);
                    else if (with_lo) ns_box_row(sbox + kNsBox, lane, low);
                }
                if (plain) {   // 64 consecutive bytes of a row of O at a time
                    __syncwarp();
                    if (col + lane < a.n) {
                        const int rows = min(32, a.m - row0);
                        for (int q = 0; q < rows; ++q)
                            reinterpret_cast<uint16_t*>(a.O)[((long long)t.mat * a.m + row0 + q) * a.n + col + lane] =
                                *reinterpret_cast<const uint16_t*>(box + q * 64 + (((lane >> 3) ^ ((q >> 1) & 3)) << 4) +
                                                                   (lane & 7) * 2);
                    }
                }
                fence_proxy_async_cta();
                __syncwarp();
                if (lane == 0) {
                    if (!plain && !plain_flip) {
                        if (flip) tma_store_3d(&tmC, box, row0, col, t.mat);
                        else tma_store_3d(&tmC, box, col, row0, t.mat);
                        if (twin) tma_store_3d(&tmC, box + kNsBox, row0, col, t.mat);
                        else if (with_lo) tma_store_3d(&tmD, box + kNsBox, col, row0, t.mat);
                    }
                    bulk_commit();
                    if (kLoads && !a.withhold_loads) {
                        bulk_wait_read<1>();   // the chunk before this one has left its slot, the next to be filled
                        request();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && rank == 1) mbar_arrive_cluster(tempty + acc, 0);
                else mbar_arrive(tempty + acc);
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) {
            bulk_wait_all();   // the stores are complete before the CTA exits, and (bounded) the loads
            for (uint32_t i = loaded > kNsSlots ? loaded - kNsSlots : 0; i < loaded; ++i)
                ns_wait_drain(box_full + i % kNsSlots, (i / kNsSlots) & 1);
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

// ---- matrices of up to 128 rows: the whole operator in one kernel --------------------------------------
// The products of a matrix with m <= 128 are too small to be launches of their own (17 of them took
// 120 us at 128 x 2048).  A cluster of CTAs takes a matrix, each CTA 256 of its columns, from G to O: X in
// fp32 registers (a thread has a row's 128 columns) and its fp16 copy in shared memory, where the rows of
// 64 columns that GRAM reads along K are, unchanged, what APPLY reads along N.  Per step:
//   partial A over the CTA's columns -> the cluster's sum, each CTA adding the rows it owns in the CTAs'
//   order and sending them to all as fp16 -> A A and B in every CTA -> X of the CTA's columns.
// B enters as fp16 and its rounding error as in the large kernels.
constexpr int kSmallCols = 256;
constexpr int kSmallThreads = 256;   // eight warps: TMEM lane quarter w % 4, column half w / 4
constexpr int kSmallX = 4 * 16384;   // X: four chunks of 128 rows x 64 columns (128-byte swizzle)
constexpr int kSmallA = 2 * 16384;   // A likewise; the partial A in fp32, later B and its rounding error
constexpr int kSmallBytes = 1024 + kSmallX + 3 * kSmallA + 256;

struct NsSmall {
    int R, C, m, n, steps, flip;
    float eps;
    float co[3 * MOE_ORTHOGONALISE_MAX_STEPS];
    __nv_bfloat16* O;
    int* status;
    long long wait_limit;
    int withhold;
};

// 16-byte chunk q (of eight) of row r in a 128-byte-swizzled chunk of 64 fp16 columns
__device__ __forceinline__ uint32_t ns_sw(int r, int q) { return (uint32_t)(r * 128 + ((q ^ (r & 7)) << 4)); }

template <typename T, bool VEC>
__global__ void __launch_bounds__(kSmallThreads, 1) ns_small_kernel(const T* __restrict__ G, const NsSmall a) {
    grid_dep_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sX = smem;
    uint8_t* sA = sX + kSmallX;
    uint8_t* sP = sA + kSmallA;                 // fp32 [128][128], then B (fp16) and its rounding error
    uint64_t* done = reinterpret_cast<uint64_t*>(sP + 2 * kSmallA);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    float* warp_sums = reinterpret_cast<float*>(tslot + 2);   // [8]
    float* my_sum = warp_sums + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = (int)gridDim.x, rank = S > 1 ? (int)cluster_ctarank() : 0, mat = blockIdx.y;
    const int quarter = warp & 3, half = warp >> 2;
    const int i = quarter * 32 + lane;                        // row of X
    const int col0 = rank * kSmallCols + half * 128;          // first of the thread's 128 columns
    if (threadIdx.x == 0) {
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    float x[128];
    float sq = 0.f;
    const T* g = G + (long long)mat * a.R * a.C;
    if (VEC && !a.flip) {
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
            if (i < a.m && col0 + j < a.n) {
                ns_val8(x + j, g + (long long)i * a.C + col0 + j);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) x[j + q] = 0.f;
            }
        }
    } else {
        const long long ri = a.flip ? 1 : a.C, rj = a.flip ? a.C : 1;
#pragma unroll
        for (int j = 0; j < 128; ++j) x[j] = i < a.m && col0 + j < a.n ? ns_val(g, i * ri + (col0 + j) * rj) : 0.f;
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
    sq = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sq += warp_sums[w];
    if (S > 1) {
        if (threadIdx.x == 0) *my_sum = sq;
        cluster_sync();
        sq = 0.f;
        for (int b = 0; b < S; ++b) sq += ld_cluster_f32(cluster_addr(my_sum, b));
    }
    float is;
    const float f = ns_split(sqrtf(sq), a.eps, &is) * kXScale;
#pragma unroll
    for (int j = 0; j < 128; ++j) x[j] *= f;

    const uint32_t bX = smem_u32(sX), bA = smem_u32(sA), bP = smem_u32(sP);
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t tA = tmem, tP = tmem + 128, tX = tmem + 256;
    const int kx = min(4, max(0, (a.n - rank * kSmallCols + 63) / 64));   // chunks of X that hold columns
    const int km = (a.m + 15) / 16;                                       // MMA steps along m
    constexpr uint32_t kIdM = idesc_f16(128, 128, false, false), kIdX = idesc_f16(128, 256, false, true);
    uint32_t phase = 0;
    // every thread after its product's commit; on a wait that ran out the rest goes through without waiting,
    // so that the CTAs of a cluster stay in step
    auto wait_mma = [&] {
        mbar_wait(done, phase, abort_flag, a.status, a.wait_limit);
        phase ^= 1u;
        __syncwarp();
        tc_fence_after();
    };
    auto put_x = [&] {   // X as fp16
#pragma unroll
        for (int j = 0; j < 128; j += 8)
            st_shared_v4(bX + (2 * half + j / 64) * 16384 + ns_sw(i, (j & 63) >> 3),
                         make_uint4(ns_pack_half(x[j], x[j + 1]), ns_pack_half(x[j + 2], x[j + 3]),
                                    ns_pack_half(x[j + 4], x[j + 5]), ns_pack_half(x[j + 6], x[j + 7])));
    };
    put_x();
    for (int s = 0; s < a.steps; ++s) {
        const float ca = a.co[3 * s], cb = a.co[3 * s + 1], cc = a.co[3 * s + 2];
        const float fa = kABScale / (kXScale * kXScale) * is * is;
        fence_proxy_async_all();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (threadIdx.x == 0 && !a.withhold) {
            for (int c = 0; c < kx; ++c)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t d = sdesc_sw128(bX + c * 16384 + ks * 32, 16, 1024);
                    mma_bf16(tA, d, d, kIdM, (c | ks) != 0);
                }
            mma_commit(done);
        }
        wait_mma();
        if (S == 1) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v[32];
                tmem_ld32(tA + lane_addr + 64 * half + 32 * c, v);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(bA + half * 16384 + ns_sw(i, 4 * c + q),
                                 make_uint4(ns_pack_half(v[8 * q] * fa, v[8 * q + 1] * fa),
                                            ns_pack_half(v[8 * q + 2] * fa, v[8 * q + 3] * fa),
                                            ns_pack_half(v[8 * q + 4] * fa, v[8 * q + 5] * fa),
                                            ns_pack_half(v[8 * q + 6] * fa, v[8 * q + 7] * fa)));
            }
        } else {
            // fp32 rows of 512 bytes, their 16-byte pieces rotated by the row against bank conflicts
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v[32];
                tmem_ld32(tA + lane_addr + 64 * half + 32 * c, v);
                const bool any = kx > 0;   // a CTA past the last column adds nothing
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int at = 16 * half + 8 * c + q;
                    st_shared_v4(bP + i * 512 + ((at ^ lane) << 4),
                                 any ? make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                                  __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]))
                                     : make_uint4(0, 0, 0, 0));
                }
            }
            cluster_sync();
            const int rows = 128 / S;
            for (int e = threadIdx.x; e < rows * 32; e += kSmallThreads) {
                const int r = rank * rows + (e >> 5), at = e & 31;
                const uint32_t off = (uint32_t)(r * 512 + ((at ^ (r & 31)) << 4));
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int b = 0; b < S; ++b) {
                    const float4 v = ld_cluster_f32x4(cluster_addr(sP, b) + off);
                    sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
                }
                const uint32_t h0 = ns_pack_half(sum.x * fa, sum.y * fa), h1 = ns_pack_half(sum.z * fa, sum.w * fa);
                const uint32_t to = (uint32_t)((at >> 4) * 16384) + ns_sw(r, (at & 15) >> 1) + (at & 1) * 8;
                for (int b = 0; b < S; ++b) st_cluster_v2(cluster_addr(sA, b) + to, h0, h1);
            }
            fence_proxy_async_all();
            cluster_sync();   // A is whole in every CTA, and the partial sums have been read
        }
        fence_proxy_async_all();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (threadIdx.x == 0 && !a.withhold) {
            for (int ks = 0; ks < km; ++ks) {
                const uint64_t d = sdesc_sw128(bA + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024);
                mma_bf16(tP, d, d, kIdM, ks != 0);
            }
            mma_commit(done);
        }
        wait_mma();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float v[32];
            tmem_ld32(tP + lane_addr + 64 * half + 32 * c, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t to = half * 16384 + ns_sw(i, 4 * c + q);
                const uint4 h = ld_shared_v4(bA + to);
                const uint32_t w[4] = {h.x, h.y, h.z, h.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 A = ns_unpack_half(w[e]);
                    const float b0 = cb * A.x + cc / kABScale * v[8 * q + 2 * e], b1 = cb * A.y + cc / kABScale * v[8 * q + 2 * e + 1];
                    hi[e] = ns_pack_half(b0, b1);
                    const float2 r = ns_unpack_half(hi[e]);
                    lo[e] = ns_pack_half(b0 - r.x, b1 - r.y);
                }
                st_shared_v4(bP + to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                st_shared_v4(bP + kSmallA + to, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
        }
        fence_proxy_async_all();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (threadIdx.x == 0 && !a.withhold) {
            for (int part = 0; part < 2; ++part)
                for (int ks = 0; ks < km; ++ks)
                    mma_bf16(tX, sdesc_sw128(bP + part * kSmallA + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024),
                             sdesc_sw128(bX + ks * 2048, 16384, 1024), kIdX, (part | ks) != 0);
            mma_commit(done);
        }
        wait_mma();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld32(tX + lane_addr + 128 * half + 32 * c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[32 * c + j] = is * (ca * x[32 * c + j] + v[j] * (1.f / kABScale));
        }
        is = 1.f;
        if (s + 1 < a.steps) put_x();
    }
    // O as it stands (16 bytes of a row at a time) or flipped (a warp's rows are 64 consecutive bytes of O)
    if (i < a.m) {
        if (a.flip) {
#pragma unroll
            for (int j = 0; j < 128; ++j)
                if (col0 + j < a.n)
                    a.O[((long long)mat * a.n + col0 + j) * a.m + i] = __float2bfloat16_rn(x[j] * (1.f / kXScale));
        } else {
            __nv_bfloat16* o = a.O + ((long long)mat * a.m + i) * a.n + col0;
#pragma unroll
            for (int j = 0; j < 128; j += 8) {
                if (VEC) {
                    if (col0 + j < a.n) {
                        constexpr float u = 1.f / kXScale;
                        *reinterpret_cast<uint4*>(o + j) =
                            make_uint4(pack_bf16x2(x[j] * u, x[j + 1] * u), pack_bf16x2(x[j + 2] * u, x[j + 3] * u),
                                       pack_bf16x2(x[j + 4] * u, x[j + 5] * u), pack_bf16x2(x[j + 6] * u, x[j + 7] * u));
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (col0 + j + q < a.n) o[j + q] = __float2bfloat16_rn(x[j + q] * (1.f / kXScale));
                }
            }
        }
    }
    // an MMA whose wait ran out may still be at work (bounded): it ends before its memory is given up
    if (*abort_flag && threadIdx.x == 0 && !a.withhold) ns_wait_drain(done, phase ^ 1u);
    tc_fence_before();
    __syncthreads();
    if (S > 1) cluster_sync();   // no CTA's shared memory is read or written any more
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- launches --------------------------------------------------------------------------------------
// CTAs of a cluster for a matrix that ns_small_kernel takes, 0 for one that it does not
static int ns_small_cluster(int64_t m, int64_t n) {
    if (m > 128) return 0;
    int S = 1;
    while (S * kSmallCols < n) S *= 2;
    return S <= 8 ? S : 0;
}

struct NsLayout {
    int64_t N, m, n, lda, ldx, parts;
    bool b_lo;
    size_t partial, inv_s, A, B, x0, x1, lo, total;
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
    if (ns_small_cluster(L->m, L->n)) {
        L->total = o;
        return true;
    }
    L->partial = take((size_t)N * L->parts * 4);
    L->inv_s = take((size_t)N * 4);
    L->A = take((size_t)N * L->m * L->lda * 2);
    L->b_lo = L->m <= 128;
    L->B = take((size_t)N * (L->b_lo ? 2 : 1) * L->m * L->lda * 2);
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

template <int MODE, bool PAIR>
static cudaError_t ns_gemm(cudaStream_t st, int num_sms, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tx,
                           const CUtensorMap& tl, const CUtensorMap& tc, const CUtensorMap& td, const NsArgs& a) {
    constexpr size_t smem = kNsSmem;
    auto kern = ns_gemm_kernel<MODE, PAIR>;
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    static int most = 0;    // resident CTAs
    std::call_once(once, [&] {
        attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        most = num_sms;
        if (attr_err == cudaSuccess && PAIR) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = 2;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(num_sms / 2 * 2);
            cfg.blockDim = dim3(kNsThreads);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int clusters = 0;
            attr_err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
            most = 2 * std::max(1, std::min(clusters, num_sms / 2));
        }
    });
    if (attr_err != cudaSuccess) return attr_err;
    if (!PAIR) return launch_pdl(kern, std::min(a.units, most), kNsThreads, smem, st, ta, tb, tx, tl, tc, td, a);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * std::min(a.units, most / 2));
    cfg.blockDim = dim3(kNsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, ta, tb, tx, tl, tc, td, a);
}

template <typename T, bool VEC>
static cudaError_t ns_small(cudaStream_t st, const T* G, int S, int N, const NsSmall& a) {
    auto kern = ns_small_kernel<T, VEC>;
    static const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallBytes);
    if (err != cudaSuccess) return err;
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
    return cudaLaunchKernelEx(&cfg, kern, G, a);
}

template <typename T>
static cudaError_t ns_first_x(cudaStream_t st, const NsLayout& L, const T* G, int R, int C, float eps, char* w, bool lo) {
    float* partial = reinterpret_cast<float*>(w + L.partial);
    const long long elems = (long long)R * C;
    const unsigned N = (unsigned)L.N;
    const dim3 parts((unsigned)L.parts, N);
    cudaError_t err = elems % 8 == 0
                          ? launch_pdl(ns_norm_kernel<T, true>, parts, 256, 0, st, G, elems, (int)L.parts, partial)
                          : launch_pdl(ns_norm_kernel<T, false>, parts, 256, 0, st, G, elems, (int)L.parts, partial);
    if (err != cudaSuccess) return err;
    const NsPrep p{partial, reinterpret_cast<__half*>(w + L.x0), lo ? reinterpret_cast<__half*>(w + L.lo) : nullptr,
                   reinterpret_cast<float*>(w + L.inv_s), (int)L.parts, R, C, (int)L.ldx, eps, R > C};
    if (C % 8 != 0) return launch_pdl(ns_prep_any_kernel<T>, dim3((C + 31) / 32, (R + 31) / 32, N), 256, 0, st, G, p);
    if (R > C) return launch_pdl(ns_prep_flip_kernel<T>, dim3((C + 63) / 64, (R + 63) / 64, N), 256, 0, st, G, p);
    return launch_pdl(ns_prep_kernel<T>, dim3((unsigned)((elems + 8 * 256 * kPrepPer - 1) / (8 * 256 * kPrepPer)), N), 256, 0, st,
                      G, p);
}

cudaError_t launch_orthogonalise(cudaStream_t st, const void* G, bool g_f32, int64_t N, int64_t R, int64_t C, void* O,
                                 int steps, const float* coeffs, float eps, void* workspace, int num_sms, int* status,
                                 long long wait_limit, bool withhold_loads) {
    NsLayout L;
    if (!ns_layout(N, R, C, &L)) return cudaErrorInvalidValue;
    if (const int S = ns_small_cluster(L.m, L.n)) {
        NsSmall a{(int)R, (int)C, (int)L.m, (int)L.n, steps, R > C, eps};
        std::copy(coeffs, coeffs + 3 * steps, a.co);
        a.O = static_cast<__nv_bfloat16*>(O);
        a.status = status;
        a.wait_limit = wait_limit > 0 ? wait_limit : kWaitTimeoutCycles;
        a.withhold = withhold_loads;
        const auto* gf = static_cast<const float*>(G);
        const auto* gb = static_cast<const __nv_bfloat16*>(G);
        if (C % 8 == 0) return g_f32 ? ns_small<float, true>(st, gf, S, (int)N, a) : ns_small<__nv_bfloat16, true>(st, gb, S, (int)N, a);
        return g_f32 ? ns_small<float, false>(st, gf, S, (int)N, a) : ns_small<__nv_bfloat16, false>(st, gb, S, (int)N, a);
    }
    char* w = static_cast<char*>(workspace);
    cudaError_t err = g_f32 ? ns_first_x(st, L, static_cast<const float*>(G), (int)R, (int)C, eps, w, steps > 1)
                            : ns_first_x(st, L, static_cast<const __nv_bfloat16*>(G), (int)R, (int)C, eps, w, false);
    if (err != cudaSuccess) return err;
    const bool flip = R > C;
    const int64_t m = L.m, n = L.n;
    char* X[2] = {w + L.x0, w + L.x1};
    // operand maps: K-major boxes of 128 rows, and 64 x 64 for X as APPLY's second operand; "s": the
    // epilogues' boxes
    CUtensorMap a_k, b_k, x_k[2], x_n[2], a_s, b_s, bl_s, x_s[2], lo_s, o_s;
    bool ok = tmap_batched(&a_k, w + L.A, false, m, m, L.lda, N, 64, 128) &&
              tmap_batched(&b_k, w + L.B, false, m, m, L.lda, L.b_lo ? 2 * N : N, 64, 128) &&
              tmap_batched(&a_s, w + L.A, false, m, m, L.lda, N, 32, 32) &&
              tmap_batched(&b_s, w + L.B, false, m, m, L.lda, N, 32, 32) &&
              tmap_batched(&bl_s, w + L.B + (L.b_lo ? (size_t)N * m * L.lda * 2 : 0), false, m, m, L.lda, N, 32, 32) &&
              tmap_batched(&lo_s, w + L.lo, false, n, m, L.ldx, N, 32, 32);
    for (int i = 0; i < 2; ++i)
        ok = ok && tmap_batched(&x_k[i], X[i], false, n, m, L.ldx, N, 64, 128) &&
             tmap_batched(&x_n[i], X[i], false, n, m, L.ldx, N, 64, 64) &&
             tmap_batched(&x_s[i], X[i], false, n, m, L.ldx, N, 32, 32);
    const bool o_box = C % 8 == 0;   // O's rows are multiples of 16 bytes
    if (o_box) ok = ok && tmap_batched(&o_s, O, true, C, R, C, N, 32, 32);
    if (!ok) return cudaErrorInvalidValue;
    NsArgs a{};
    a.m = (int)m; a.n = (int)n; a.lda = (int)L.lda; a.ldx = (int)L.ldx;
    a.batch = (int)N;
    a.status = status;
    a.wait_limit = wait_limit > 0 ? wait_limit : kWaitTimeoutCycles;
    a.withhold_loads = withhold_loads;
    a.O = static_cast<__nv_bfloat16*>(O);
    const bool pair = m > 128 && N * ((m + 255) / 256) * ((n + 255) / 256) >= num_sms / 2;
    const int tile = pair ? 256 : 128;
    const int mt = (int)((m + tile - 1) / tile), nt = (int)((n + tile - 1) / tile);
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        const bool last = s + 1 == steps;
        a.a = coeffs[3 * s]; a.b = coeffs[3 * s + 1]; a.c = coeffs[3 * s + 2];
        a.inv_s = s == 0 ? reinterpret_cast<float*>(w + L.inv_s) : nullptr;
        a.tiles = mt * (mt + 1) / 2;
        a.units = (int)N * a.tiles;
        a.k_blocks = a.k_wrap = (int)((n + 63) / 64);
        a.keep_lo = 0;
        a.out_kind = NS_O_NONE;
        err = pair ? ns_gemm<NS_GRAM, true>(st, num_sms, x_k[cur], x_k[cur], a_s, a_s, a_s, a_s, a)
                   : ns_gemm<NS_GRAM, false>(st, num_sms, x_k[cur], x_k[cur], a_s, a_s, a_s, a_s, a);
        if (err != cudaSuccess) return err;
        a.k_blocks = a.k_wrap = (int)((m + 63) / 64);
        a.keep_lo = L.b_lo;
        err = pair ? ns_gemm<NS_POLY, true>(st, num_sms, a_k, a_k, a_s, a_s, b_s, bl_s, a)
                   : ns_gemm<NS_POLY, false>(st, num_sms, a_k, a_k, a_s, a_s, b_s, bl_s, a);
        if (err != cudaSuccess) return err;
        if (L.b_lo) a.k_blocks = 2 * a.k_wrap;
        a.tiles_n = nt;
        a.tiles = mt * nt;
        a.units = (int)N * a.tiles;
        a.xlo = (s == 0 ? g_f32 && !last : !last);
        a.keep_lo = s + 2 < steps;   // the last step reads no rounding error, so the one before it keeps none
        if (last) a.out_kind = o_box ? (flip ? NS_O_BOX_FLIP : NS_O_BOX) : (flip ? NS_O_PLAIN_FLIP : NS_O_PLAIN);
        const CUtensorMap& out = last ? (o_box ? o_s : x_s[1 - cur]) : x_s[1 - cur];
        err = pair ? ns_gemm<NS_APPLY, true>(st, num_sms, b_k, x_n[cur], x_s[cur], lo_s, out, lo_s, a)
                   : ns_gemm<NS_APPLY, false>(st, num_sms, b_k, x_n[cur], x_s[cur], lo_s, out, lo_s, a);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace moe
