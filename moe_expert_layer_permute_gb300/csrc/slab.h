// slab.h - which elements of a matrix each CTA of ns_small_kernel (orthogonal.cu) copies, and in which words;
// plain C++ as well, so that the copies' bounds are checked on the host for every kind of size
// (tests/test_orthogonalise_copies.py).
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

constexpr int kSmallCols = 256;      // columns of one block of X
constexpr int kSmallThreads = 256;   // eight warps: TMEM lane quarter w % 4, column half w / 4

// CTAs of a cluster for matrices that ns_small_kernel takes, 0 for others, and the rows of a block.  Up to 64 rows
// it takes any number of matrices, since the large kernel's tiles have 128 (200 matrices of 40 x 4096: 692 us
// here, 1052 there; 64 x 2000, 300: 421 and 815); so do one or two CTAs, and four whose columns are filled
// (100 x 1000, 200: 316 and 378; 128 x 1024, 256: 434 and 472).  Of more CTAs the kernel runs about 57 us a round
// of the GPU however few the matrices are, and the large kernel is even with it beyond 512 CTAs if filled, and at
// two rounds of the SMs if not (128 x 2048, 40, 64, 128 matrices: 176, 290, 528 us here and 231, 284, 455 there;
// 128 x 4096, 32 and 64: 334, 666 and 361, 559; 70 x 600, 76 and 128: 142, 193 and 127, 163).
inline int ns_small_cluster(int64_t N, int64_t m, int64_t n, int* mp) {
    *mp = 128;
    while (*mp / 2 >= m && *mp > 16 && (128 / *mp) * kSmallCols < n) *mp /= 2;
    const int cols = 128 / *mp * kSmallCols;
    if (m > 128 || n > 16 * cols) return 0;
    int S = 1;
    while (S * cols < n) S *= 2;
    const bool filled = 4 * n > 3 * S * cols;
    return *mp < 128 || S <= 2 || (S == 4 && filled) || N * S <= (filled ? 512 : 304) ? S : 0;
}

// A CTA's part of G comes in, and O goes out, through shared memory where G^T is kept or rows are no multiples
// of 16 bytes (16 x 128 x 255, bf16: 34 us; by single elements of each row it was 34 us more; 16 x 128 x 256, 32 us with
// rows of 16-byte pieces, which threads take from G themselves, was 1 us more this way).  A part is a run of all
// the CTA's columns, which are G's rows (flip), or for each row of each block of columns one of up to 256
// elements, `pitch` bytes apart in shared memory: an odd number of words, so that threads of consecutive rows
// meet no bank conflicts.  Copies are of words of W bytes, aligned on both sides: the data lies as far past a word in
// shared memory as it does in global memory, words that it begins within come whole and go by elements.  A CTA
// whose columns begin past the last one (the CTAs of a cluster are a power of two) has empty runs: no copies.
struct NsRun {
    int first, at, count;   // first element of the matrix, offset in shared memory, elements
};
struct NsSlab {
    int m, n, log_mp, flip, cta0;   // cta0: the CTA's first column of X
    MOE_HD NsRun columns() const {   // flip
        const int held = n - cta0, most = (128 >> log_mp) * kSmallCols;
        return {cta0 * m, 0, held <= 0 ? 0 : (held < most ? held : most) * m};
    }
    MOE_HD NsRun row(int r, int pitch) const {   // row r of the CTA's 128 (128 n < 2^31)
        const int i = r & ((1 << log_mp) - 1), c = cta0 + (r >> log_mp) * kSmallCols;
        const int left = n - c;
        return {i * n + c, r * pitch, i < m && left > 0 ? (left < kSmallCols ? left : kSmallCols) : 0};
    }
    // move(run) for this thread's (flip) or warp's runs, empty ones left out
    template <typename F>
    MOE_HD void each(int pitch, int warp, F move) const {
        if (flip) {
            const NsRun run = columns();
            if (run.count > 0) move(run);
            return;
        }
        // (four rows at a time: one after the other took 300 cycles each in their addresses alone)
#ifdef __CUDACC__
#pragma unroll 4
#endif
        for (int k = 0; k < 128 / (kSmallThreads / 32); ++k) {
            const NsRun run = row(warp + k * (kSmallThreads / 32), pitch);
            if (run.count > 0) move(run);
        }
    }
};
// The words of W bytes that hold `bytes` bytes from `from` on: the first one's address, and where the data
// begins and ends past it; `copy(offset, bytes of the word that hold data or what is before it)` for thread t's.
template <int W>
struct NsWords {
    uintptr_t at;
    int begin, end;
    MOE_HD NsWords(uintptr_t from, int bytes) : at(from & ~uintptr_t(W - 1)), begin((int)(from - at)), end(begin + bytes) {}
    template <int STEP, int UNROLL, typename F>
    MOE_HD void each(int t, F copy) const {
#ifdef __CUDACC__
#pragma unroll UNROLL
#endif
        for (int w = W * t; w < end; w += W * STEP) copy(w, W < end - w ? W : end - w);
    }
};

}  // namespace moe
