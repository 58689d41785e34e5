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
constexpr int kNsTile = 128;       // output tile
constexpr int kNsStages = 3;
constexpr int kNsThreads = 192;    // TMA, MMA, four epilogue warps
constexpr int kNsOperand = kNsTile * 128;   // bytes of one operand's K slice: 128 x 64 fp16
constexpr int kNormPart = 32768;   // elements of one partial sum of squares
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

template <typename T>
__global__ void __launch_bounds__(256) ns_norm_kernel(const T* G, long long elems, int parts, float* partial) {
    grid_dep_wait();
    const long long base = (long long)blockIdx.y * elems;
    float v = 0.f;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < elems; i += (long long)parts * 256) {
        const float g = ns_val(G, base + i);
        v += g * g;
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

// 32 x 32 tiles through shared memory, so that both the plain and the flipped copy are coalesced
template <typename T>
__global__ void __launch_bounds__(256) ns_prep_kernel(const T* G, const NsPrep a) {
    grid_dep_wait();
    __shared__ float tile[32][33];
    const int mat = blockIdx.z;
    float v = 0.f;
    for (int i = threadIdx.x; i < a.parts; i += 256) v += a.partial[(long long)mat * a.parts + i];
    float inv_s;
    const float f = ns_split(sqrtf(ns_block_sum(v)), a.eps, &inv_s) * kXScale;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.inv_s[mat] = inv_s;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long rows = a.flip ? a.C : a.R;
    for (int r0 = blockIdx.y * 32; r0 < a.R; r0 += gridDim.y * 32) {
        const int c0 = blockIdx.x * 32;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            const int r = r0 + ty + j, c = c0 + tx;
            tile[ty + j][tx] = r < a.R && c < a.C ? ns_val(G, ((long long)mat * a.R + r) * a.C + c) * f : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            const int r = a.flip ? c0 + ty + j : r0 + ty + j, c = a.flip ? r0 + tx : c0 + tx;
            if (r >= rows || c >= (a.flip ? a.R : a.C)) continue;
            const float x = a.flip ? tile[tx][ty + j] : tile[ty + j][tx];
            const __half h = __float2half_rn(x);
            const long long at = ((long long)mat * rows + r) * a.ld + c;
            a.hi[at] = h;
            if (a.lo) a.lo[at] = __float2half_rn((x - __half2float(h)) * kLoScale);
        }
    }
}

// ---- the three products ------------------------------------------------------------------------------
enum NsMode { NS_GRAM = 0, NS_POLY, NS_APPLY };

struct NsArgs {
    int m, n, lda, ldx, k_blocks, tiles_n, tiles;   // tiles per matrix
    int k_wrap;                  // k_blocks, or half of them: APPLY with B's rounding error as a second B
    int batch;                   // N: matrix N + i of the B array is the rounding error of matrix i's B
    float a, b, c;
    const float* inv_s;          // [N] in the first step, null after it
    const __half* A;             // POLY: reads its tile of A
    __half* out;                 // GRAM: A, POLY: B, APPLY: next X
    __half* out_lo;              // POLY: B's rounding error (null: not kept)
    const __half* xhi;           // APPLY: this X
    const __half* xlo;           // APPLY: its rounding error (null: exact)
    __half* xlo_out;             // APPLY: the next X's rounding error (null: not kept)
    __nv_bfloat16* O;            // APPLY, last step: the result
    int flip;                    // O is [n, m]
    int* status;
    long long wait_limit;
    int withhold_loads;
};

__device__ __forceinline__ void ns_wait_drain(uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kDrainCycles) break;
}

// One 128 x 128 tile per block.  GRAM and POLY are symmetric: tiles of the lower triangle alone, each
// stored twice.  Operands: GRAM rows of X by rows of X, POLY rows of A by rows of A (A = A^T), both
// contiguous along K; APPLY rows of B by columns of X (contiguous along N).
// K past the edge is zero-filled by the TMA.
template <int MODE>
__global__ void __launch_bounds__(kNsThreads) ns_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                                                            const __grid_constant__ CUtensorMap tmB, const NsArgs a) {
    grid_dep_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kNsStages * kNsOperand;
    uint64_t* full = reinterpret_cast<uint64_t*>(sB + kNsStages * kNsOperand);
    uint64_t* empty = full + kNsStages;
    uint64_t* done = empty + kNsStages;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mat = blockIdx.x / a.tiles, tile = blockIdx.x - mat * a.tiles;
    int ti, tj;
    if (MODE == NS_APPLY) {
        ti = tile / a.tiles_n;
        tj = tile - ti * a.tiles_n;
    } else {
        ti = 0;
        int left = tile;
        while (left > ti) left -= ++ti;   // row ti of the triangle has ti + 1 tiles
        tj = left;
    }
    const int m0 = ti * kNsTile, n0 = tj * kNsTile;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kNsStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tslot, kNsTile);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    constexpr bool kBmn = MODE == NS_APPLY;
    constexpr uint32_t kIdesc = idesc_f16(kNsTile, kNsTile, false, kBmn);

    if (warp == 0) {
        if (lane == 0 && !a.withhold_loads) {
            int issued = 0;
            for (int kb = 0; kb < a.k_blocks; ++kb) {
                const int st = kb % kNsStages;
                if (!mbar_wait(empty + st, ((kb / kNsStages) & 1) ^ 1u, abort_flag, a.status, a.wait_limit)) break;
                mbar_arrive_expect_tx(full + st, 2 * kNsOperand);
                const int k0 = (kb < a.k_wrap ? kb : kb - a.k_wrap) * 64;
                tma_load_3d(sA + st * kNsOperand, &tmA, full + st, k0, m0, kb < a.k_wrap ? mat : mat + a.batch);
                if (kBmn) {
                    tma_load_3d(sB + st * kNsOperand, &tmB, full + st, n0, k0, mat);
                    tma_load_3d(sB + st * kNsOperand + 64 * 128, &tmB, full + st, n0 + 64, k0, mat);
                } else {
                    tma_load_3d(sB + st * kNsOperand, &tmB, full + st, k0, n0, mat);
                }
                ++issued;
            }
            // the block does not exit before its copies have landed (bounded), whoever gave up
            for (int s = 0; s < kNsStages; ++s)
                if (issued > s) ns_wait_drain(full + s, (uint32_t)(((issued - s + kNsStages - 1) / kNsStages - 1) & 1));
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            for (int kb = 0; kb < a.k_blocks; ++kb) {
                const int st = kb % kNsStages;
                if (!mbar_wait(full + st, (kb / kNsStages) & 1, abort_flag, a.status, a.wait_limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(sA) + st * kNsOperand, sb = smem_u32(sB) + st * kNsOperand;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem, sdesc_sw128(sa + ks * 32, 16, 1024),
                             kBmn ? sdesc_sw128(sb + ks * 2048, 64 * 128, 1024) : sdesc_sw128(sb + ks * 32, 16, 1024),
                             kIdesc, (kb | ks) != 0);
                mma_commit(empty + st);
            }
            mma_commit(done);
            if (!ok) ns_wait_drain(done, 0);
        }
    } else if (__all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag, a.status, a.wait_limit) && !*abort_flag)) {
        tc_fence_after();
        const int quarter = warp & 3;
        const int r = m0 + quarter * 32 + lane;
        const float is = a.inv_s ? __ldg(a.inv_s + mat) : 1.f;
        const long long row = (long long)mat * a.m + r;
#pragma unroll 1
        for (int c0 = 0; c0 < kNsTile; c0 += 32) {
            float v[32];
            __syncwarp();
            tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + c0, v);
            const int col = n0 + c0;
            if (r >= a.m) continue;
            if (MODE != NS_APPLY) {
                if (MODE == NS_GRAM) {
                    const float f = kABScale / (kXScale * kXScale) * is * is;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= f;
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = col + j < a.m ? a.b * __half2float(a.A[row * a.lda + col + j]) + a.c / kABScale * v[j] : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (col + j >= a.m) continue;
                    const __half h = __float2half_rn(v[j]);
                    a.out[row * a.lda + col + j] = h;
                    if (ti != tj) a.out[((long long)mat * a.m + col + j) * a.lda + r] = h;
                    // (kept for a single tile only)
                    if (MODE == NS_POLY && a.out_lo) a.out_lo[row * a.lda + col + j] = __float2half_rn(v[j] - __half2float(h));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (col + j >= a.n) continue;
                    const long long at = row * a.ldx + col + j;
                    float x = __half2float(a.xhi[at]);
                    if (a.xlo) x += __half2float(a.xlo[at]) * (1.f / kLoScale);
                    x = is * (a.a * x + v[j] * (1.f / kABScale));
                    if (a.O) {
                        const long long o = a.flip ? ((long long)mat * a.n + col + j) * a.m + r : row * a.n + col + j;
                        a.O[o] = __float2bfloat16_rn(x * (1.f / kXScale));
                    } else {
                        const __half h = __float2half_rn(x);
                        a.out[at] = h;
                        if (a.xlo_out) a.xlo_out[at] = __float2half_rn((x - __half2float(h)) * kLoScale);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kNsTile);
    }
}

// ---- launches --------------------------------------------------------------------------------------
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
    L->partial = take((size_t)N * L->parts * 4);
    L->inv_s = take((size_t)N * 4);
    L->A = take((size_t)N * L->m * L->lda * 2);
    L->b_lo = L->m <= kNsTile;
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

// 3-D map of a batch of row-major [rows, cols] fp16 matrices with pitch ld; box 64 columns x box_rows.
// Reads outside a matrix are zero.
static bool ns_tmap(CUtensorMap* m, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int64_t N, int box_rows) {
    return tmap_batched_f16(m, ptr, (uint64_t)cols, (uint64_t)rows, (uint64_t)ld, (uint64_t)N, (uint32_t)box_rows);
}

template <int MODE>
static cudaError_t ns_gemm(cudaStream_t st, const CUtensorMap& ta, const CUtensorMap& tb, const NsArgs& a, int64_t N) {
    constexpr size_t smem = 1024 + 2 * kNsStages * kNsOperand + 256;
    static const cudaError_t err =
        cudaFuncSetAttribute(ns_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    return launch_pdl(ns_gemm_kernel<MODE>, (unsigned)(N * a.tiles), kNsThreads, smem, st, ta, tb, a);
}

template <typename T>
static cudaError_t ns_first_x(cudaStream_t st, const NsLayout& L, const T* G, int R, int C, float eps, char* w, bool lo) {
    float* partial = reinterpret_cast<float*>(w + L.partial);
    cudaError_t err = launch_pdl(ns_norm_kernel<T>, dim3((unsigned)L.parts, (unsigned)L.N), 256, 0, st, G, (long long)R * C,
                                 (int)L.parts, partial);
    if (err != cudaSuccess) return err;
    NsPrep p{partial, reinterpret_cast<__half*>(w + L.x0), lo ? reinterpret_cast<__half*>(w + L.lo) : nullptr,
             reinterpret_cast<float*>(w + L.inv_s), (int)L.parts, R, C, (int)L.ldx, eps, R > C};
    return launch_pdl(ns_prep_kernel<T>, dim3((C + 31) / 32, std::min((R + 31) / 32, 32), (unsigned)L.N), 256, 0, st, G, p);
}

cudaError_t launch_orthogonalise(cudaStream_t st, const void* G, bool g_f32, int64_t N, int64_t R, int64_t C, void* O,
                                 int steps, const float* coeffs, float eps, void* workspace, int* status,
                                 long long wait_limit, bool withhold_loads) {
    NsLayout L;
    if (!ns_layout(N, R, C, &L)) return cudaErrorInvalidValue;
    char* w = static_cast<char*>(workspace);
    cudaError_t err = g_f32 ? ns_first_x(st, L, static_cast<const float*>(G), (int)R, (int)C, eps, w, steps > 1)
                            : ns_first_x(st, L, static_cast<const __nv_bfloat16*>(G), (int)R, (int)C, eps, w, false);
    if (err != cudaSuccess) return err;
    CUtensorMap ta, tb, tx[2], txn[2];
    for (int i = 0; i < 2; ++i)
        if (!ns_tmap(&tx[i], w + (i ? L.x1 : L.x0), L.n, L.m, L.ldx, N, kNsTile) ||
            !ns_tmap(&txn[i], w + (i ? L.x1 : L.x0), L.n, L.m, L.ldx, N, 64))
            return cudaErrorInvalidValue;
    if (!ns_tmap(&ta, w + L.A, L.m, L.m, L.lda, N, kNsTile) || !ns_tmap(&tb, w + L.B, L.m, L.m, L.lda, L.b_lo ? 2 * N : N, kNsTile))
        return cudaErrorInvalidValue;
    const int mt = (int)((L.m + kNsTile - 1) / kNsTile), nt = (int)((L.n + kNsTile - 1) / kNsTile);
    NsArgs a{};
    a.m = (int)L.m; a.n = (int)L.n; a.lda = (int)L.lda; a.ldx = (int)L.ldx;
    a.batch = (int)N;
    a.status = status;
    a.wait_limit = wait_limit > 0 ? wait_limit : kWaitTimeoutCycles;
    a.withhold_loads = withhold_loads;
    a.A = reinterpret_cast<__half*>(w + L.A);
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        const bool last = s + 1 == steps;
        a.a = coeffs[3 * s]; a.b = coeffs[3 * s + 1]; a.c = coeffs[3 * s + 2];
        a.inv_s = s == 0 ? reinterpret_cast<float*>(w + L.inv_s) : nullptr;
        a.tiles = mt * (mt + 1) / 2;
        a.k_blocks = a.k_wrap = (int)((L.n + 63) / 64);
        a.out = reinterpret_cast<__half*>(w + L.A);
        if ((err = ns_gemm<NS_GRAM>(st, tx[cur], tx[cur], a, N)) != cudaSuccess) return err;
        a.inv_s = nullptr;
        a.k_blocks = a.k_wrap = (int)((L.m + 63) / 64);
        a.out = reinterpret_cast<__half*>(w + L.B);
        a.out_lo = L.b_lo ? a.out + (size_t)N * L.m * L.lda : nullptr;
        if ((err = ns_gemm<NS_POLY>(st, ta, ta, a, N)) != cudaSuccess) return err;
        a.inv_s = s == 0 ? reinterpret_cast<float*>(w + L.inv_s) : nullptr;
        a.k_blocks = L.b_lo ? 2 * a.k_wrap : a.k_wrap;
        a.tiles_n = nt;
        a.tiles = mt * nt;
        a.xhi = reinterpret_cast<__half*>(w + (cur ? L.x1 : L.x0));
        a.xlo = (s == 0 ? g_f32 && !last : !last) ? reinterpret_cast<__half*>(w + L.lo) : nullptr;
        // the last step reads no rounding error, so the one before it keeps none
        a.xlo_out = s + 2 < steps ? reinterpret_cast<__half*>(w + L.lo) : nullptr;
        a.out = reinterpret_cast<__half*>(w + (cur ? L.x0 : L.x1));
        a.O = last ? static_cast<__nv_bfloat16*>(O) : nullptr;
        a.flip = R > C;
        if ((err = ns_gemm<NS_APPLY>(st, tb, txn[cur], a, N)) != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace moe
