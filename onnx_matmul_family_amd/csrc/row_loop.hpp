// Building blocks of K loops over operands that are both read along their rows
// (16x16 MFMAs, gemm16_core.hpp), with any number of stages in LDS: more of them
// keep the matrix unit fed where tiles are small or few.
#pragma once
#include "gemm16_core.hpp"

namespace omm {
namespace core16 {

// R rows of an operand, 128 bytes a stage, by DMA: the layout of DmaSrc's K-major
// tile.  Rows past the last are out of the buffer's range and read as zeros.
// KT: so are the 16-byte pieces of a row past its end (ends: its bytes, a multiple of
// 16); without it the last stage reads on into the next row.
template <int R, bool KT = false, int WAVES = 4>
struct RowSrc {
    static constexpr int PER_WAVE = R / 8 / WAVES;
    static_assert(PER_WAVE % 2 == 0, "block parity == parity of the wave-local block index");
    const char* base;
    uint32_t ldb, bytes, ends;
    uint32_t lane_off[2], piece[2];
    // row_bytes: from one row to the next; R row_bytes < 2 GiB
    __device__ __forceinline__ void init(const void* p, uint32_t row_bytes, uint32_t ends_, int64_t row0, int64_t rows, int lane) {
        ldb = row_bytes;
        ends = ends_;
        base = (const char*)p + row0 * ldb;
        bytes = (uint32_t)min((int64_t)R, rows - row0) * ldb;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            piece[q] = (uint32_t)(((lane & 7) ^ kswz(8 * q + (lane >> 3))) << 4);
            lane_off[q] = (uint32_t)(lane >> 3) * ldb + piece[q];
        }
    }
    // begin with stage kt
    __device__ __forceinline__ void skip(int kt) {
        base += (int64_t)kt * 128;
        bytes -= (uint32_t)kt * 128u;
    }
    // (a stage past the last: an empty range)
    __device__ __forceinline__ i32x4_t rsrc(int kt, int nk) const {
        i32x4_t r = make_rsrc(base + (kt < nk ? kt * 128 : 0));
        r.z = __builtin_amdgcn_readfirstlane(kt < nk ? (int)(bytes - (uint32_t)kt * 128u) : 0);
        return r;
    }
    // block j of this wave's share of stage kt
    __device__ __forceinline__ void one(const i32x4_t& r, uint32_t lds, int kt, int wave, int j) const {
        const int b = wave * PER_WAVE + j;
        uint32_t off = lane_off[j & 1] + (uint32_t)(b * 8) * ldb;
        if constexpr (KT) off = (uint32_t)kt * 128u + piece[j & 1] < ends ? off : DMA_OOB;
        dma16u(r, lds + b * 1024, off);
    }
};

// One phase: the products of fragments a x b into acc, step(x) after the x-th
template <int DT, int TM, int TN, bool Z, class F>
__device__ __forceinline__ void phase(f32x4_t (&acc)[TM][TN], const u32x4_t (&a)[TM], const u32x4_t (&b)[TN], F&& step) {
    static_for<0, TM * TN>([&](auto xc) {
        constexpr int x = decltype(xc)::value;
        mfma16_tied<DT, Z>(acc[x / TN][x % TN], b[x % TN], a[x / TN]);
        step(xc);
        fence_sched();
    });
}
// n things over the steps of a phase of N: f(i) for those due after step x
template <int N, int n, int x, class F>
__device__ __forceinline__ void spread(F&& f) {
    static_for<(x * n + N - 1) / N, ((x + 1) * n + N - 1) / N>(f);
}

// acc_fence for 2 or 6 column blocks
template <int TM>
__device__ __forceinline__ void acc_fence(f32x4_t (&acc)[TM][2]) {
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3" : "+a"(acc[i][0]), "+a"(acc[i][1]));
}
template <int TM>
__device__ __forceinline__ void acc_fence(f32x4_t (&acc)[TM][6]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3"
                     : "+a"(acc[i][0]), "+a"(acc[i][1]), "+a"(acc[i][2]), "+a"(acc[i][3]), "+a"(acc[i][4]), "+a"(acc[i][5]));
}

// Tile size of a launch, by what was measured (us): a tile's own time beside its
// stages, a stage where the chip is nearly idle, one where every CU has a tile
// (`alone`), and one where every place is taken (`full`; two places a CU where two
// workgroups fit one).
struct TileTimes {
    int bt, places;
    double own, idle, alone, full;
};
inline double tile_time(const TileTimes& t, int64_t n, double stages) {
    const int64_t rest = n % t.places;
    double time = (double)(n / t.places) * (t.own + stages * t.full);
    if (rest > 256) time += t.own + stages * t.full;
    else if (rest) time += t.own + stages * (t.idle + (t.alone - t.idle) * (double)rest / 256);
    return time;
}
// tiles(bt): how many there are
template <size_t N, class F>
int pick_tile(const TileTimes (&times)[N], double stages, F&& tiles) {
    int best = 0;
    double least = 0.0;
    for (const TileTimes& t : times) {
        const double time = tile_time(t, tiles(t.bt), stages);
        if (!best || time < least) {
            best = t.bt;
            least = time;
        }
    }
    return best;
}

}  // namespace core16
}  // namespace omm
