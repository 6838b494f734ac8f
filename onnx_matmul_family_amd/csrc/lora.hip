// A shared projection with low-rank adapters chosen per row:
//   Y[m] = X[m] W (+ bias) + scale[g] (X[m] A[g]) B[g],   g = idx[m]
// (a row whose g is outside [0, G) has no adapter).
//
// Here: the streamed form by groups of 64 rows (T = scale X A on the vector ALU,
// then X W streamed once a group with T B added), and an element-wise form for
// what it does not take.  One row, 4096 x 4096, rank 16 (bf16, trans 1): 3.2 + 6.5
// us, W at 5.2 TB/s from the last-level cache; 43 rows of 32 adapters, 4096 x
// 4104, rank 24 (fp16, trans 0): 4.4 + 22 us, where W takes 7 and the join of the
// K parts with its round trips as long.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.hpp"
#include "lora_args.hpp"
#include "row_select.hpp"
#include "stream_core.hpp"

namespace omm {

namespace {

// T[p, r] = scale[g] sum_k X[m, k] A[g, k, r], m the row at position p: a
// workgroup a row, a wave an r.
template <int DT>
__global__ __launch_bounds__(256) void lora_shrink_any_kernel(LoraK a) {
    typedef typename elem_of<DT>::type E;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t p = blockIdx.x, m = a.perm ? a.perm[p] : p, g = row_adapter(a, m);
    if (g < 0) return;
    const E* x = (const E*)a.X + m * a.K;
    const int64_t sk = a.trans ? 1 : a.R, sr = a.trans ? a.K : 1;
    for (int r = wave; r < a.R; r += 4) {
        const E* w = (const E*)a.A + g * a.K * a.R + r * sr;
        float acc = 0.0f;
        for (int64_t k = lane; k < a.K; k += 64) acc = fmaf(elem_f32<DT>(x[k]), elem_f32<DT>(w[k * sk]), acc);
        acc = wave_sum(acc);
        if (lane == 0) a.T[p * a.R + r] = a.scale ? acc * a.scale[g] : acc;
    }
}

// Y[m, n] = bias[n] + sum_r T[m, r] B[g, r, n]
template <int DT>
__global__ __launch_bounds__(256) void lora_delta_any_kernel(LoraK a, int64_t nblk) {
    typedef typename elem_of<DT>::type E;
    const int64_t m = blockIdx.x / nblk, n = (blockIdx.x - m * nblk) * 256 + threadIdx.x;
    if (n >= a.N) return;
    const int64_t g = row_adapter(a, m);
    float acc = a.bias ? elem_f32<DT>(((const E*)a.bias)[n]) : 0.0f;
    if (g >= 0) {
        const int64_t sr = a.trans ? 1 : a.N, sn = a.trans ? a.R : 1;
        const E* b = (const E*)a.B + g * a.R * a.N + n * sn;
        const float* t = a.T + m * a.R;
        for (int r = 0; r < a.R; ++r) acc = fmaf(t[r], elem_f32<DT>(b[r * sr]), acc);
    }
    ((E*)a.Y)[m * a.N + n] = f32_elem<DT>(acc);
}

// ------------------------------------------------------------------ few rows (at most 64)
// T[m, r] = scale[g] sum_k X[m, k] A[g, k, r], some workgroups a row: the rows of
// a decode batch have adapters of their own, so A is read once a row whatever
// the tiling, on the vector ALU; one CU takes in 32 bytes a clock or so, hence
// the shares of 32 to 64 KiB.
//   TRANS = 1: a wave an r, 16 bytes of k a lane.
//   TRANS = 0: a workgroup a quarter of K (its sum in T's quarter; the reader
//     adds them up); a thread takes V columns of every (512 / tpr)-th k (tpr
//     threads a row of R, a power of two); sums over k by shuffles, then LDS.
// It also zeroes the counters of the kernel that follows it.
template <int TRANS> constexpr int kParts = TRANS ? 1 : 4;

template <int DT, int TRANS, int V>
__global__ __launch_bounds__(TRANS ? 256 : 512) void lora_shrink_kernel(LoraK a, int tpr) {
    typedef typename elem_of<DT>::type E;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.y == 0 && blockIdx.x == 0)
        for (int64_t i = tid; i < (a.M + 63) / 64 * ((a.N + a.cw - 1) / a.cw); i += blockDim.x) a.done[i] = 0;
    row_group(a, blockIdx.y >> 6, kParts<TRANS>, sizeof(E));
    const int64_t m = blockIdx.y & 63;
    const int64_t g = row_adapter(a, m);
    if (g < 0 || a.R == 0) return;
    const E* x = (const E*)a.X + m * a.K;
    const float scale = a.scale ? a.scale[g] : 1.0f;
    const int K = (int)a.K;
    if constexpr (TRANS) {
        const int r = blockIdx.x * 4 + wave;
        if (r >= a.R) return;
        const E* w = (const E*)a.A + (g * a.R + r) * a.K;
        float acc = 0.0f;
        const int kv = K / V;
        // U loads of each on their way at once (past the end: the last one, not used)
        constexpr int U = 8;
        for (int c0 = lane; c0 < kv; c0 += 64 * U) {
            u32x4_t xr[U], wr[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = min(c0 + 64 * u, kv - 1) * V;
                xr[u] = load16(x + c);
                wr[u] = load16(w + c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + 64 * u >= kv) continue;
                float xv[V], wv[V];
                unpack16<DT>(xr[u], xv);
                unpack16<DT>(wr[u], wv);
#pragma unroll
                for (int i = 0; i < V; ++i) acc = fmaf(xv[i], wv[i], acc);
            }
        }
        const int k = kv * V + lane;
        if (k < K) acc = fmaf(elem_f32<DT>(x[k]), elem_f32<DT>(w[k]), acc);
        acc = wave_sum(acc);
        if (lane == 0) a.T[m * a.R + r] = acc * scale;
    } else {
        __shared__ float red[8][64][V];
        const int rb = tid & (tpr - 1), kk = tid / tpr, kn = 512 / tpr;
        const int kc = (K + kParts<0> - 1) / kParts<0>, kb = blockIdx.x * kc, ke = min(K, kb + kc);
        const int start = min(rb * V, a.R - V);  // the last group may overlap the one before
        const bool mine = rb * V < a.R;
        float acc[V] = {};
        if (mine) {
            const E* w = (const E*)a.A + g * a.K * a.R + start;
            constexpr int U = 8;
            for (int k0 = kb + kk; k0 < ke; k0 += U * kn) {
                E xr[U];
                u32x4_t wr[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = min(k0 + u * kn, ke - 1);
                    xr[u] = x[k];
                    if constexpr (V == 1)
                        wr[u][0] = __builtin_bit_cast(uint32_t, elem_f32<DT>(w[(int64_t)k * a.R]));
                    else
                        wr[u] = load16(w + (int64_t)k * a.R);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (k0 + u * kn >= ke) continue;
                    const float xv = elem_f32<DT>(xr[u]);
                    float wv[V];
                    if constexpr (V == 1)
                        wv[0] = __uint_as_float(wr[u][0]);
                    else
                        unpack16<DT>(wr[u], wv);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = fmaf(xv, wv[i], acc[i]);
                }
            }
        }
        for (int d = tpr; d < 64; d <<= 1)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += __shfl_xor(acc[i], d, 64);
        if (lane < tpr)
#pragma unroll
            for (int i = 0; i < V; ++i) red[wave][lane][i] = acc[i];
        __syncthreads();
        if (tid < a.R) {
            const int b = tid / V, i = tid - min(b * V, a.R - V);
            float v = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += red[u][b][i];
            a.T[(blockIdx.x * a.M + m) * a.R + tid] = v * scale;
        }
    }
}

// ex[j][c] = sum_r T[m, r] B[g, r, c0 + c] of the rows m = split + j splits.
//   TRANS = 1: a thread a column, 16 bytes of r a load.
//   TRANS = 0: a thread 16 bytes of columns, one r a load.
template <int DT, int TRANS, int CW>
__device__ __forceinline__ void lora_expand(const LoraK& a, int split, int c0, float (*ex)[CW], int tid) {
    typedef typename elem_of<DT>::type E;
    constexpr int V = kQ<DT>, TPR = TRANS ? CW : CW / V;  // threads a row
    const int M = (int)a.M, N = (int)a.N, R = a.R;
    const int c = TRANS ? tid & (CW - 1) : (tid & (TPR - 1)) * V;
    if (c0 + c >= N) return;
    const int n = TRANS ? c0 + c : group_start<DT>(c0, c, N);
    for (int j = tid / TPR, m = split + j * a.splits; m < M; j += 512 / TPR, m = split + j * a.splits) {
        const int64_t g = row_adapter(a, m);
        const float* t = a.T + m * R;
        const E* b = (const E*)a.B + (g < 0 ? 0 : g) * R * a.N + (TRANS ? (int64_t)n * R : n);
        const int rn = g < 0 ? 0 : R, rv = rn / V * V;
        if constexpr (TRANS) {
            float acc = 0.0f;
#pragma unroll 4
            for (int r = 0; r < rv; r += V) {
                float bv[V];
                unpack16<DT>(load16(b + r), bv);
#pragma unroll
                for (int i = 0; i < V; ++i) acc = fmaf(t[r + i], bv[i], acc);
            }
            for (int r = rv; r < rn; ++r) acc = fmaf(t[r], elem_f32<DT>(b[r]), acc);
            ex[j][c] = acc;
        } else {
            float acc[V] = {};
            const auto tsum = [&](const float* p) {
                float v = p[0];
#pragma unroll
                for (int u = 1; u < kParts<TRANS>; ++u) v += p[(int64_t)u * M * R];
                return v;
            };
            const auto row = [&](u32x4_t w, float tv) {
                float bv[V];
                unpack16<DT>(w, bv);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(tv, bv[i], acc[i]);
            };
            int r = 0;
            for (; r + 8 <= rn; r += 8) {
                u32x4_t w[8];
                float tv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[i] = load16(b + (int64_t)(r + i) * a.N);
                    tv[i] = tsum(t + r + i);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) row(w[i], tv[i]);
            }
            for (; r < rn; ++r) row(load16(b + (int64_t)r * a.N), tsum(t + r));
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (n + i >= c0 + c) ex[j][n + i - c0] = acc[i];
        }
    }
}

// Y of 128 columns: X W streamed (8 waves split the workgroup's part of K),
// the adapters' share of the rows m = split mod splits, and, in the last
// workgroup of the columns to finish, the sum over the parts.
template <int DT, int TRANS, int NG>
__global__ __launch_bounds__(512, 2) void lora_stream_kernel(LoraK a) {
    typedef typename elem_of<DT>::type E;
    row_group(a, blockIdx.z, kParts<TRANS>, sizeof(E));
    __shared__ __attribute__((aligned(16))) float red[8 * 8 * kFragPad];
    __shared__ float ex[16 * NG][128];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15;
    const int q = (lane >> 4) * kQ<DT>, tr = x_row<TRANS>(lane), tq = x_off<DT, TRANS>(lane), sp = blockIdx.y;
    const int M = (int)a.M, K = (int)a.K, N = (int)a.N, c0 = blockIdx.x * 128;
    StreamW<DT, TRANS> w;
    const E* wp = (const E*)a.W;
    if constexpr (TRANS) {
        w.base[0] = w.base[1] = wp;
#pragma unroll
        for (int j = 0; j < 8; ++j) w.off[j] = (uint32_t)min(c0 + 16 * j + tr, N - 1) * K + tq;
    } else {
        w.ld = N;
        if constexpr (DT == 2) {
            w.p[0] = wp + group_start<DT>(c0, 4 * i, N) + (int64_t)q * N;
            w.p[1] = wp + group_start<DT>(c0, 64 + 4 * i, N) + (int64_t)q * N;
        } else {
            w.p[0] = wp + group_start<DT>(c0, 8 * i, N) + (int64_t)q * N;
        }
    }
    StreamX<DT, TRANS, NG> x;  // rows past the last are the last one: their results are not used
#pragma unroll
    for (int g = 0; g < NG; ++g) x.p[g] = (const E*)a.X + (int64_t)min(16 * g + tr, M - 1) * K + tq;
    f32x4_t acc[8][NG] = {};
    int s0, s1;
    wave_steps<DT, 8>(K, TRANS, wave, s0, s1, a.splits, sp);
    stream_run<DT, TRANS, NG>(w, x, s0, s1, K, acc, (u32x4_t*)&red[red_index(wave, 0, 0, 0)], lane, [&] { lora_expand<DT, TRANS, 128>(a, sp, c0, ex, tid); });
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g) __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) *(f32x4_t*)&red[red_index(wave, j, lane, 0)] = acc[j][g];
        __syncthreads();
        for (int o = tid; o < 16 * 128; o += 512) {
            const int c = o & 127, row = o >> 7, m = 16 * g + row;
            const int n = c0 + c;
            if (m >= M || n >= N) continue;
            int j, l, rr;
            red_pos<DT, TRANS>(c, c0 + (c & ~(kQ<DT> - 1)) - group_start<DT>(c0, c, N), row, j, l, rr);
            float v = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += red[red_index(u, j, l, rr)];
            if (m % a.splits == sp) v += ex[m / a.splits][c];
            if (a.splits == 1) {
                if (a.bias) v += elem_f32<DT>(((const E*)a.bias)[n]);
                ((E*)a.Y)[(int64_t)m * N + n] = f32_elem<DT>(v);
            } else {
                part_store<128>(a.part, ((int64_t)blockIdx.x * a.splits + sp) * M + m, c, v);
            }
        }
    }
    // (the kernel before this one zeroed the count)
    if (a.splits == 1 || !part_last(&a.done[blockIdx.x], a.splits, tid)) return;
    part_sums<512, 128>(
        a.part, M, a.splits, tid, [&](int m, int p) { return ((int64_t)blockIdx.x * a.splits + p) * M + m; },
        [&](int m, int c, float v0, float v1) {
            const int n = c0 + c;
            E* y = (E*)a.Y + (int64_t)m * N + n;
            if (n < N) y[0] = f32_elem<DT>(v0 + (a.bias ? elem_f32<DT>(((const E*)a.bias)[n]) : 0.0f));
            if (n + 1 < N) y[1] = f32_elem<DT>(v1 + (a.bias ? elem_f32<DT>(((const E*)a.bias)[n + 1]) : 0.0f));
        });
}

// Y of 16 NF columns, otherwise as lora_stream_kernel.
template <int DT, int TRANS, int NG, int NF, int U>
__global__ __launch_bounds__(512, 2) void lora_cols_kernel(LoraK a) {
    typedef typename elem_of<DT>::type E;
    row_group(a, blockIdx.z, kParts<TRANS>, sizeof(E));
    constexpr int CW = 16 * NF, TILES = NF > NG ? NF : NG;
    constexpr int RED = 8 * NF * NG * kFragPad, SCR = 8 * TILES * 256;
    __shared__ __attribute__((aligned(16))) float red[RED > SCR ? RED : SCR];
    __shared__ float ex[16 * NG][CW];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int M = (int)a.M, K = (int)a.K, N = (int)a.N;
    // (blocks split evenly over the XCDs, a run of neighbours each)
    const int bx = blockIdx.x & 7, block = bx * (int)(gridDim.x >> 3) + min(bx, (int)(gridDim.x & 7)) + (blockIdx.x >> 3);
    const int c0 = block * CW, sp = blockIdx.y;
    u32x4_t* scratch = (u32x4_t*)&red[wave * TILES * 256];
    ColsWeights<DT, TRANS, NF> w;
    cols_start<DT, TRANS, NF>(w, (const E*)a.W, c0, N, K, lane);
    StreamX<DT, 1, NG> x;  // rows past the last are the last one: their results are not used
#pragma unroll
    for (int g = 0; g < NG; ++g) x.p[g] = (const E*)a.X + (int64_t)min(16 * g + tile_row(lane), M - 1) * K + tile_off<DT>(lane);
    f32x4_t acc[NF][NG] = {};
    int s0, s1;
    wave_steps<DT, 8>(K, 1, wave, s0, s1, a.splits, sp);
    cols_run<DT, TRANS, NG, NF, U>(w, x, s0, s1, K, acc, scratch, lane,
                                   [&] { lora_expand<DT, TRANS, CW>(a, sp, c0, ex, tid); });
    __syncthreads();  // (the image overlaps other waves' scratch)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int g = 0; g < NG; ++g) *(f32x4_t*)&red[((wave * NF + j) * NG + g) * kFragPad + lane * 4] = acc[j][g];
    __syncthreads();
    for (int o = tid; o < M * CW; o += 512) {
        const int c = o % CW, m = o / CW, n = c0 + c;
        if (n >= N) continue;
        const int pos = cols_pos<DT, TRANS>(c0, c, N);
        const float* p = &red[((pos >> 4) * NG + (m >> 4)) * kFragPad + (((pos & 15) >> 2) * 16 + (m & 15)) * 4 + (pos & 3)];
        float v = m % a.splits == sp ? ex[m / a.splits][c] : 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) v += p[u * NF * NG * kFragPad];
        if (a.splits == 1)
            ((E*)a.Y)[(int64_t)m * N + n] = f32_elem<DT>(v + (a.bias ? elem_f32<DT>(((const E*)a.bias)[n]) : 0.0f));
        else
            part_store<CW>(a.part, ((int64_t)block * a.splits + sp) * M + m, c, v);
    }
    // (the kernel before this one zeroed the count)
    if (a.splits == 1 || !part_last(&a.done[block], a.splits, tid)) return;
    part_sums<512, CW>(
        a.part, M, a.splits, tid, [&](int m, int p) { return ((int64_t)block * a.splits + p) * M + m; },
        [&](int m, int c, float v0, float v1) {
            const int n = c0 + c;
            E* y = (E*)a.Y + (int64_t)m * N + n;
            if (n < N) y[0] = f32_elem<DT>(v0 + (a.bias ? elem_f32<DT>(((const E*)a.bias)[n]) : 0.0f));
            if (n + 1 < N) y[1] = f32_elem<DT>(v1 + (a.bias ? elem_f32<DT>(((const E*)a.bias)[n + 1]) : 0.0f));
        });
}

constexpr int64_t kFew = 64;  // rows a group

// How the streamed forms share the work: columns of a workgroup (128:
// lora_stream_kernel, fewer: lora_cols_kernel) and the parts that K is split
// into.  Fewer columns make more workgroups without splitting K, whose parts
// must be joined by the last one (its time grows with rows and parts), but read
// X more often.  Measured at K = 4096, bf16, W from memory, us with 16 / 32 / 64
// / 128 columns:
//   trans 1   N = 1024, 43 rows    8.8   10.7  12.2  18.2
//             N = 2056,  1 row     8.9   10.4  10.0  10.6;  43 rows  16.5  14.2  15.5  21.0
//             N = 4104,  1 row    16.7   14.5  16.2  16.8;  43 rows  28.0  22.9  22.2  27.4
//             N = 8200,  1 row    29.4   30.5  27.8  26.0;  64 rows  52.8  52.2  43.0  62.8
//   trans 0   N = 1024,  1 row    10.7   10.7   8.9  10.1;  43 rows  12.1  12.2  13.6  18.3
//             N = 2056,  1 row    14.7   12.7  12.4  10.7;  43 rows  19.4  16.7  17.9  19.5
//             N = 4104,  1 row    20.2   18.6  16.7  13.5;  43 rows  31.9  26.1  22.4  23.2
//             N = 8200, 43 rows   50.7   42.3  39.7  35.9
// So trans 1 (whose columns are rows of memory, any number is as good): as few
// as leave 256 column blocks, one a CU (N = 4104, 16 / 32 columns: 1 row 14.9 / 13.7, 16
// rows 18.0 / 16.1), over 16 rows 72.  trans 0: wide ones unless N is
// small.  K goes into as many parts as fill 256 CUs, each wave two steps of 32 or
// more (of the counts that leave a wave the same steps, the smallest), but in
// one where up to 16 rows already make 100 workgroups (1 row, trans 1, N = 2048:
// 9.0 against 10.6 us with two parts, from the last-level cache 5.6 against 6.2).
struct StreamPlan {
    int cw, splits;
};
StreamPlan stream_plan(int64_t M, int64_t K, int64_t N, int trans) {
    StreamPlan p;
    const bool few = M <= 16;
    if (trans) {
        const int64_t most = few ? 256 : 72;
        p.cw = N <= 16 * most ? 16 : N <= 32 * most ? 32 : N <= 64 * most || !few ? 64 : 128;
    } else if (few) {
        p.cw = N <= 1152 ? 64 : 128;
    } else {
        p.cw = N <= 16 * 72 ? 16 : N <= 32 * 72 ? 32 : 128;
    }
    const int64_t groups = (N + p.cw - 1) / p.cw * ((M + kFew - 1) / kFew), steps = (K + 31) / 32;
    int64_t s = few && p.cw < 128 && groups >= 100 ? 1 : 256 / groups;
    if (s > steps / 16) s = steps / 16;
    if (s > 16) s = 16;
    if (s < 1) s = 1;
    const int64_t per = (steps + 8 * s - 1) / (8 * s);
    p.splits = (int)((steps + 8 * per - 1) / (8 * per));
    return p;
}
// (the workspace does not depend on the layout: the larger of both)
size_t part_bytes(int64_t M, int64_t K, int64_t N) {
    size_t most = 0;
    for (int trans = 0; trans < 2; ++trans) {
        const StreamPlan p = stream_plan(M, K, N, trans);
        const size_t n = p.splits > 1 ? (size_t)p.splits * M * ((N + p.cw - 1) / p.cw) * p.cw * 4 : 0;
        if (n > most) most = n;
    }
    return most;
}

// whole groups of 8 columns, W within 32-bit byte offsets
bool streamable(int64_t K, int64_t N, int dt) {
    return K >= 8 && N >= 8 && K * N < (dt == 2 ? 1LL << 29 : 1LL << 30);
}

// Rows of one launch of each form; a call of more is taken in pieces, one after
// the other in the same workspace (bf16 and fp16: the forms that add the adapter's
// term to a dense product round it to T before the sum).
//   streamed: a row a grid index in y.
//   tiles: 32-bit byte offsets into X (any other form of lora_rows.hip: as many);
//     all of them within 2^32 threads.
//   element-wise: 2^32 threads of 256 columns.
constexpr int64_t kStreamRows = 1023 * kFew;
constexpr int64_t kMaxBlocks = (1 << 24) - 1;
int64_t tile_rows(int64_t K, int64_t N, int dt) {
    int64_t n = 1 << 20;
    const int64_t offsets = dt < 2 && K > 0 ? ((1LL << 31) - 1) / (2 * K) : n;
    if (offsets >= 256) n = std::min(n, offsets);  // (else no tiles)
    n = std::min(n, kMaxBlocks / ((N + 127) / 128) * 128);
    return std::max<int64_t>(n / 256 * 256, 128);
}
int64_t any_rows(int64_t N) { return std::max<int64_t>(1, kMaxBlocks / ((N + 255) / 256)); }
// M rows in pieces of at most `most`: rows of a piece (the last one may have fewer)
int64_t piece_rows(int64_t M, int64_t most) {
    const int64_t n = (M + most - 1) / most, even = (M + n - 1) / n;
    return std::min(most, (even + 255) / 256 * 256);
}

// Where the streamed form (W once per 64 rows, mostly from the caches) is ahead
// of the tiles over sorted rows, or of the dense product after the adapters'
// term where there are no tiles.  us a call, streamed / other (bf16, rank 16):
//   K, N (trans)         M = 256     M = 512      M = 1024     M = 2048
//   4096, 1024 (1)     17 /  48     32 /  58     58 /  59    107 /  61
//   4096, 4096 (1)     31 /  58     58 /  59    110 /  62    208 /  78
//   4096, 8192 (1)     55 /  60    112 /  61    205 /  76    403 / 120
//   1175, 3329 (1)     35 / 133     67 / 188    124 / 180    222 / 218   (no tiles)
//   4000, 8190 (0)     47 / 423     85 / 427    161 / 605    312 / 1174  (no tiles)
bool stream_ahead(int64_t M, int64_t K, int64_t N, bool tiles) {
    if (M <= 256) return true;
    return tiles ? M <= 512 && K * N <= 1 << 24 : true;
}

// (steps on their way a register set: as many as fit)
template <int DT, int TRANS, int NF>
void cols_launch(const LoraK& a, int ng, dim3 grid, hipStream_t s) {
    switch (ng) {
        case 1: return lora_cols_kernel<DT, TRANS, 1, NF, NF == 4 ? 2 : 4><<<grid, 512, 0, s>>>(a);
        case 2: return lora_cols_kernel<DT, TRANS, 2, NF, NF == 4 ? 2 : 4><<<grid, 512, 0, s>>>(a);
        case 3: return lora_cols_kernel<DT, TRANS, 3, NF, NF == 1 ? 4 : 2><<<grid, 512, 0, s>>>(a);
        default: return lora_cols_kernel<DT, TRANS, 4, NF, 2><<<grid, 512, 0, s>>>(a);
    }
}

template <int DT, int TRANS>
void lora_streamed(const LoraK& a, hipStream_t s) {
    constexpr int V = kQ<DT>;
    if constexpr (TRANS) {
        lora_shrink_kernel<DT, 1, V><<<dim3((unsigned)((a.R + 3) / 4 + !a.R), (unsigned)a.M), 256, 0, s>>>(a, 0);
    } else {
        const int v = a.R >= V ? V : 1;
        int tpr = 1;
        while (tpr * v < a.R) tpr *= 2;
        const dim3 grid(kParts<0>, (unsigned)a.M);
        if (v == V) lora_shrink_kernel<DT, 0, V><<<grid, 512, 0, s>>>(a, tpr);
        else lora_shrink_kernel<DT, 0, 1><<<grid, 512, 0, s>>>(a, tpr);
    }
    const dim3 grid((unsigned)((a.N + a.cw - 1) / a.cw), (unsigned)a.splits, (unsigned)((a.M + kFew - 1) / kFew));
    const int ng = a.M >= kFew ? 4 : (int)((a.M + 15) / 16);
    if constexpr (TRANS) {
        switch (a.cw) {
            case 16: return cols_launch<DT, 1, 1>(a, ng, grid, s);
            case 32: return cols_launch<DT, 1, 2>(a, ng, grid, s);
            case 64: return cols_launch<DT, 1, 4>(a, ng, grid, s);
            default: return lora_stream_kernel<DT, 1, 1><<<grid, 512, 0, s>>>(a);  // (up to 16 rows)
        }
    } else {
        switch (a.cw) {
            case 16: return cols_launch<DT, 0, 1>(a, ng, grid, s);
            case 32: return cols_launch<DT, 0, 2>(a, ng, grid, s);
            case 64: return lora_cols_kernel<DT, 0, 1, 4, 2><<<grid, 512, 0, s>>>(a);  // (up to 16 rows)
            default: break;
        }
        switch (ng) {
            case 1: return lora_stream_kernel<DT, 0, 1><<<grid, 512, 0, s>>>(a);
            case 2: return lora_stream_kernel<DT, 0, 2><<<grid, 512, 0, s>>>(a);
            case 3: return lora_stream_kernel<DT, 0, 3><<<grid, 512, 0, s>>>(a);
            default: return lora_stream_kernel<DT, 0, 4><<<grid, 512, 0, s>>>(a);
        }
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// of one piece (the form depends on layout and alignment too: room for each)
static size_t piece_bytes(int64_t M, int64_t K, int64_t N, int64_t R, bool stream) {
    const size_t rows = M > kFew || !stream ? lora_rows_workspace_bytes(M, R) : 0;
    if (!stream || M > kStreamRows) return rows;
    const size_t groups = (size_t)(M + kFew - 1) / kFew;
    const size_t bytes = align256(groups * kFew * R * 4 * kParts<0>) + align256(part_bytes(M, K, N)) +
                         align256(groups * ((N + 15) / 16) * 4);
    return rows > bytes ? rows : bytes;
}
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R, int dt) {
    const bool stream = streamable(K, N, dt) && !(dt == 2 && M > kStreamRows);
    size_t most = 0;
    for (const int64_t limit : {kStreamRows, tile_rows(K, N, dt), any_rows(N)}) {
        const int64_t piece = piece_rows(M, limit), last = M - (M - 1) / piece * piece;
        for (const int64_t m : {piece, last}) most = std::max(most, piece_bytes(std::min(m, M), K, N, R, stream));
    }
    return most;
}

hipError_t lora_add_dense(const LoraK& a, const void* C, int dt, hipStream_t s) {
    DenseArgs d = {};
    d.A = a.X;
    d.B = a.W;
    d.Y = a.Y;
    d.C = C;
    d.M = a.M;
    d.N = a.N;
    d.K = a.K;
    d.lda = a.K;
    d.ldb = a.trans ? a.K : a.N;
    d.ldy = a.N;
    d.nb0 = d.nb1 = 1;
    d.c_sm = a.N;
    d.c_sn = 1;
    d.alpha = 1.0f;
    d.beta = 1.0f;
    d.a_kmajor = 1;
    d.b_kmajor = a.trans;
    return dt == 2 ? launch_dense_f32(d, s) : launch_dense16(d, dt, s);
}

void lora_shrink_any(const LoraK& a, int dt, hipStream_t s) {
    const dim3 grid((unsigned)a.M);
    if (dt == 0) lora_shrink_any_kernel<0><<<grid, 256, 0, s>>>(a);
    else if (dt == 1) lora_shrink_any_kernel<1><<<grid, 256, 0, s>>>(a);
    else lora_shrink_any_kernel<2><<<grid, 256, 0, s>>>(a);
}

// one piece
static hipError_t launch_piece(LoraK a, int dt, bool stream, bool rows, void* ws, hipStream_t s) {
    if (stream && (!rows || stream_ahead(a.M, a.K, a.N, lora_tiles_ok(a, dt)))) {
        const StreamPlan p = stream_plan(a.M, a.K, a.N, a.trans);
        a.splits = p.splits;
        a.cw = p.cw;
        a.part = (float*)((char*)ws + align256((size_t)(a.M + kFew - 1) / kFew * kFew * a.R * 4 * kParts<0>));
        a.done = (uint32_t*)((char*)a.part + align256(part_bytes(a.M, a.K, a.N)));
        log_choice("lora_matmul: streamed, %d columns a workgroup, K in %d part(s)", a.cw, a.splits);
        switch (dt * 2 + a.trans) {
            case 0: lora_streamed<0, 0>(a, s); break;
            case 1: lora_streamed<0, 1>(a, s); break;
            case 2: lora_streamed<1, 0>(a, s); break;
            case 3: lora_streamed<1, 1>(a, s); break;
            case 4: lora_streamed<2, 0>(a, s); break;
            default: lora_streamed<2, 1>(a, s); break;
        }
        return hipGetLastError();
    }
    if (rows) return launch_lora_rows(a, dt, ws, s);
    log_choice("lora_matmul: element-wise");
    const int64_t nblk = (a.N + 255) / 256;
    const dim3 grid((unsigned)(a.M * nblk));
    lora_shrink_any(a, dt, s);
    if (dt == 0) lora_delta_any_kernel<0><<<grid, 256, 0, s>>>(a, nblk);
    else if (dt == 1) lora_delta_any_kernel<1><<<grid, 256, 0, s>>>(a, nblk);
    else lora_delta_any_kernel<2><<<grid, 256, 0, s>>>(a, nblk);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : lora_add_dense(a, a.Y, dt, s);
}

hipError_t launch_lora(const LoraArgs& l, int dt, void* ws, hipStream_t s) {
    LoraK a = {};
    a.X = l.X;
    a.W = l.W;
    a.A = l.A;
    a.B = l.B;
    a.idx = l.idx;
    a.scale = l.scale;
    a.bias = l.bias;
    a.Y = l.Y;
    a.T = (float*)ws;
    a.K = l.K;
    a.N = l.N;
    a.G = l.G;
    a.R = (int)l.R;
    a.trans = l.trans;
    a.idx64 = l.idx64;
    // Over 65472 rows, us a call, streamed / other (rank 16, trans 1):
    //   fp32, 65600 rows of 1024 x 1024            2974 / 1920 (adapters into Y, the dense product)
    //                       2001 x 1003            5221 / 3055
    //   bf16, 65600 rows of 1024 x 1024, rank 4,
    //         trans 0                              1856 / 481 (tiles, T by elements)
    const bool many = l.M > kStreamRows;
    const bool stream = streamable(l.K, l.N, dt) && !(dt == 2 && many);
    a.M = piece_rows(l.M, tile_rows(l.K, l.N, dt));
    const bool narrow = !l.trans && l.R > 0 && l.R < 8, tiles = lora_tiles_ok(a, dt);
    const bool rows = lora_rows_ok(l.K, l.N, l.R, l.G) && (!narrow || (many && tiles));
    const int64_t piece = rows && (tiles || !stream) ? a.M : piece_rows(l.M, stream ? kStreamRows : any_rows(l.N));
    const int64_t elem = dt == 2 ? 4 : 2;
    for (int64_t m = 0; m < l.M; m += piece) {
        a.M = std::min(piece, l.M - m);
        a.X = (const char*)l.X + m * l.K * elem;
        a.Y = (char*)l.Y + m * l.N * elem;
        a.idx = (const char*)l.idx + m * (l.idx64 ? 8 : 4);
        const hipError_t e = launch_piece(a, dt, stream, rows, ws, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace omm
