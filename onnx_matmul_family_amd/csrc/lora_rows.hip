// The projection with per-row adapters for more than 64 rows (prompts):
//   Y[m] = X[m] W (+ bias) + scale[g] (X[m] A[g]) B[g],   g = idx[m].
//
// Rows are taken in the order of their adapters (a stable counting sort, so
// that results do not depend on scheduling), which makes almost every block of
// 16 rows one of a single adapter:
//   lora_sort_kernel         the order
//   lora_shrink_rows_kernel  T = scale X A, 16 rows a workgroup, left as three
//                            16-bit parts that add up to its fp32 values
//   lora_tile_kernel         Y tiles on the LDS-DMA matrix core; as a tile
//                            leaves, T B is added to its accumulators, part by
//                            part, so neither T nor T B is rounded.
// (T is split where it is computed.  Split again in every column tile, 3844 rows of
// 512 x 4480, rank 8, trans 1, took 98 us in bf16 and 107 in fp16; now 73 and 76.)
// Operands that the DMA cannot take (rows not 16-byte aligned) and fp32, with a
// W too large for the streamed form (2 GiB and more):
//   lora_expand_kernel       bias + T B into Y, to which the framework's dense
//                            product is then added.
// A block of rows that mixes adapters multiplies each one's B on its own and
// adds it under a mask: a zero row times another adapter's infinity would be
// NaN.
#include <algorithm>

#include "gemm16_core.hpp"
#include "kernels.hpp"
#include "lora_args.hpp"
#include "stream_core.hpp"

namespace omm {

namespace {

using namespace core16;

constexpr int kSortWaves = 16;

__device__ __forceinline__ int row_of(const LoraK& a, int p) { return a.perm ? a.perm[p] : p; }

// Stable counting sort of the rows by adapter (bin 0: none) in one workgroup:
// each wave counts its contiguous share of the rows per bin, a scan over (bin,
// wave) gives every wave its place in every bin, and it writes its rows there.
// 4096 rows: 8 us in runs of 9 bins, 11 us mixed over 17; the tiles
// that use the order take 208 and up.
__global__ __launch_bounds__(64 * kSortWaves) void lora_sort_kernel(LoraK a, int bins) {
    extern __shared__ int hist[];  // [wave][bin]
    __shared__ int wsum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int M = (int)a.M, per = (((M + kSortWaves - 1) / kSortWaves) + 63) / 64 * 64;
    const int m0 = min(M, wave * per), m1 = min(M, m0 + per);
    for (int i = tid; i < kSortWaves * bins; i += 64 * kSortWaves) hist[i] = 0;
    __syncthreads();
    int* mine = hist + wave * bins;
    for (int m = m0 + lane; m < m1; m += 64) atomicAdd(&mine[row_adapter(a, m) + 1], 1);
    __syncthreads();
    // exclusive scan in the order (bin, wave); one bin a thread (bins <= 1024)
    int total = 0;
    if (tid < bins)
        for (int w = 0; w < kSortWaves; ++w) total += hist[w * bins + tid];
    int scan = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(scan, d, 64);
        if (lane >= d) scan += o;
    }
    if (lane == 63) wsum[wave] = scan;
    __syncthreads();
    for (int w = 0; w < wave; ++w) scan += wsum[w];
    scan -= total;
    if (tid < bins)
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = hist[w * bins + tid];
            hist[w * bins + tid] = scan;
            scan += n;
        }
    __syncthreads();
    for (int m = m0 + lane; m - lane < m1; m += 64) {
        const int b = m < m1 ? (int)row_adapter(a, m) + 1 : -1;
        uint64_t same = 0;  // the lanes whose row has this lane's adapter
        for (uint64_t todo = __ballot(b >= 0); todo;) {
            const uint64_t in = __ballot(b == __builtin_amdgcn_readlane(b, __ffsll((unsigned long long)todo) - 1));
            if ((in >> lane) & 1) same = in;
            todo &= ~in;
        }
        if (b >= 0) {
            const int at = mine[b], rank = __popcll(same & ((1ull << lane) - 1));
            a.perm[at + rank] = m;
            if (rank == 0) mine[b] = at + __popcll(same);
        }
    }
}

// T[p, r] = scale[g] sum_k X[m, k] A[g, k, r] of the 16 rows m at positions p0
// .. p0 + 15 and 16 NF r: NW waves split K, A and the rows go from memory
// to the matrix unit.  One pass for each adapter among the rows.  bf16 and fp16: the
// parts of T, fp16 scaled by a power of two for the 16 NF r of the row.
template <int DT, int TRANS, int NF, int NW>
__global__ __launch_bounds__(64 * NW) void lora_shrink_rows_kernel(LoraK a) {
    typedef typename elem_of<DT>::type E;
    constexpr int CW = 16 * NF;
    __shared__ __attribute__((aligned(16))) float red[NW * NF * kFragPad];
    __shared__ uint32_t max_s[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15;
    const int M = (int)a.M, K = (int)a.K, R = a.R, p0 = blockIdx.x * 16, c0 = blockIdx.y * CW;
    const int m = row_of(a, min(p0 + i, M - 1));
    const int ad = p0 + i < M ? (int)row_adapter(a, m) : -1;
    StreamX<DT, 1, 1> x;
    x.p[0] = (const E*)a.X + (int64_t)__shfl(m, tile_row(lane), 64) * K + tile_off<DT>(lane);
    if (tid < 16) max_s[tid] = 0;
    int s0, s1;
    wave_steps<DT, NW>(K, 1, wave, s0, s1);
    for (uint32_t todo = (uint32_t)__ballot(ad >= 0) & 0xffffu; todo;) {
        const int g = __builtin_amdgcn_readlane(ad, __ffs(todo) - 1);
        const uint32_t in = (uint32_t)__ballot(ad == g) & 0xffffu;
        todo &= ~in;
        ColsWeights<DT, TRANS, NF> w;
        cols_start<DT, TRANS, NF>(w, (const E*)a.A + (int64_t)g * K * R, c0, R, K, lane);
        f32x4_t acc[NF][1] = {};
        cols_run<DT, TRANS, 1, NF, NF == 1 ? 4 : 2>(w, x, s0, s1, K, acc, (u32x4_t*)&red[wave * NF * kFragPad], lane,
                                                    [] {});
#pragma unroll
        for (int j = 0; j < NF; ++j) *(f32x4_t*)&red[(wave * NF + j) * kFragPad + lane * 4] = acc[j][0];
        __syncthreads();
        const float scale = a.scale ? a.scale[g] : 1.0f;
        constexpr int NV = (16 * CW + 64 * NW - 1) / (64 * NW);  // values a thread
        float v[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int o = tid + n * 64 * NW, c = o % CW, row = o / CW;
            v[n] = 0.0f;
            if (row >= 16 || !((in >> row) & 1) || c0 + c >= R) continue;
            const int pos = cols_pos<DT, TRANS>(c0, c, R);
            const float* q = &red[(pos >> 4) * kFragPad + (((pos & 15) >> 2) * 16 + row) * 4 + (pos & 3)];
#pragma unroll
            for (int u = 0; u < NW; ++u) v[n] += q[u * NF * kFragPad];
            v[n] *= scale;
            if constexpr (DT == 2) a.T[(int64_t)(p0 + row) * R + c0 + c] = v[n];
            if constexpr (DT == 1) atomicMax(&max_s[row], __float_as_uint(fabsf(v[n])));  // (NaN is the largest)
        }
        if constexpr (DT == 1) __syncthreads();
        if constexpr (DT < 2) {
            const int rp = (R + 7) & ~7;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int o = tid + n * 64 * NW, c = o % CW, row = o / CW;
                if (row >= 16 || !((in >> row) & 1) || c0 + c >= rp) continue;
                float w = v[n], none = 0.0f;
                if constexpr (DT == 1) {
                    const int e = split_exp(__uint_as_float(max_s[row]));
                    w = split_raise<DT>(w * ldexpf(1.0f, e));
                    if (c == 0) a.undo[(int64_t)(p0 + row) * gridDim.y + blockIdx.y] = ldexpf(1.0f, -e);
                }
                uint16_t* t = a.Tp + (int64_t)(p0 + row) * rp + c0 + c;
#pragma unroll
                for (int h = 0; h < kParts32; ++h) t[h * (a.M * rp)] = (uint16_t)split_pair<DT>(w, none);
            }
        }
        if (todo) __syncthreads();
    }
}

// r of a workgroup of the kernel above, and its workgroups a row
__host__ __device__ inline int shrink_cols(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }
__host__ __device__ inline int shrink_parts(int R) { return (R + shrink_cols(R) - 1) / shrink_cols(R); }

// fp16: what the parts of position p's r from 64 b on are multiplied by
__device__ __forceinline__ float row_undo(const LoraK& a, int64_t p, int b) { return a.undo[p * shrink_parts(a.R) + b]; }

// T of up to 8 r -> its parts, a thread a position
template <int DT>
__global__ __launch_bounds__(256) void lora_split_kernel(LoraK a) {
    const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (p >= a.M) return;
    if (row_adapter(a, row_of(a, (int)p)) < 0) return;
    float v[8], mx = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        v[r] = r < a.R ? a.T[p * a.R + r] : 0.0f;
        mx = fmaxf(mx, fabsf(v[r]));
    }
    if constexpr (DT == 1) {
        const int e = split_exp(mx);
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = split_raise<DT>(v[r] * ldexpf(1.0f, e));
        a.undo[p] = ldexpf(1.0f, -e);
    }
#pragma unroll
    for (int h = 0; h < kParts32; ++h) {
        u32x4_t t;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = split_pair<DT>(v[2 * i], v[2 * i + 1]);
        *(u32x4_t*)(a.Tp + (h * a.M + p) * 8) = t;
    }
}

// Y[m, n] = bias[n] + sum_r T[p, r] B[g, r, n], a wave 16 positions and 128 columns
template <int DT, int TRANS>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraK a) {
    typedef typename elem_of<DT>::type E;
    __shared__ u32x4_t scratch[4][8 * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = (lane >> 4) * kQ<DT>;
    const int tr = x_row<TRANS>(lane), tq = x_off<DT, TRANS>(lane);
    const int M = (int)a.M, N = (int)a.N, R = a.R, c0 = blockIdx.x * 128;
    const int64_t pw = ((int64_t)blockIdx.y * 4 + wave) * 16;
    if (pw >= M) return;
    const int p = (int)min(pw + i, (int64_t)M - 1), m = row_of(a, p);
    const int ad = (int)row_adapter(a, m);
    typename std::conditional<DT == 2, StreamX<2, TRANS, 1>, StreamXParts<DT, TRANS, 1>>::type x;
    const int64_t xrow = min(pw + tr, (int64_t)M - 1);
    if constexpr (DT == 2) {
        x.p[0] = a.T + xrow * R + x.off(lane);
    } else {
        const int rp = (R + 7) & ~7;
        x.p[0] = a.Tp + xrow * rp + x.off(lane);
        x.plane = a.M * rp;
    }
    f32x4_t res[8] = {};
    for (uint32_t todo = (uint32_t)__ballot(ad >= 0) & 0xffffu; todo;) {
        const int g = __builtin_amdgcn_readlane(ad, __ffs(todo) - 1);
        todo &= ~(uint32_t)__ballot(ad == g);
        const E* B = (const E*)a.B + (int64_t)g * R * N;
        StreamW<DT, TRANS> w;
        if constexpr (TRANS) {
            w.base[0] = w.base[1] = B;
#pragma unroll
            for (int j = 0; j < 8; ++j) w.off[j] = (uint32_t)min(c0 + 16 * j + tr, N - 1) * R + tq;
        } else {
            w.ld = N;
            if constexpr (DT == 2) {
                w.p[0] = B + group_start<DT>(c0, 4 * i, N) + (int64_t)q * N;
                w.p[1] = B + group_start<DT>(c0, 64 + 4 * i, N) + (int64_t)q * N;
            } else {
                w.p[0] = B + group_start<DT>(c0, 8 * i, N) + (int64_t)q * N;
            }
        }
        // (fp16: 64 r at a time, which have a scale of their own)
        const int steps = (R + kStep<DT> - 1) / kStep<DT>, span = DT == 1 ? 2 : steps;
        for (int s0 = 0; s0 < steps; s0 += span) {
            f32x4_t acc[8][1] = {};
            stream_run<DT, TRANS, 1>(w, x, s0, min(steps, s0 + span), R, acc, scratch[wave], lane);
            const float undo = DT == 1 && ad == g ? row_undo(a, p, s0 / 2) : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) res[j][e] = ad == g ? fmaf(acc[j][0][e], undo, res[j][e]) : res[j][e];
        }
    }
    if (pw + i >= M) return;
    E* y = (E*)a.Y + (int64_t)m * N;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = (lane >> 4) * 4 + e;  // the lane's fragment column
            int n;
            if constexpr (TRANS)
                n = c0 + 16 * j + t;
            else if constexpr (DT == 2)
                n = group_start<DT>(c0, 64 * (j >> 2) + 4 * t, N) + (j & 3);
            else
                n = group_start<DT>(c0, 8 * t, N) + j;
            if (n < N) y[n] = f32_elem<DT>(res[j][e] + (a.bias ? elem_f32<DT>(((const E*)a.bias)[n]) : 0.0f));
        }
}

// BT x BT tiles of Y over the sorted rows: the dense product's K loop
// (mainloop_dma16, rows of X gathered through the order), then T B block by
// block from registers.
// BKM: W (N, K), B (G, N, R); else W (K, N), B (G, R, N).
// TH: column fragments of a pass of the epilogue; fewer (4 of 8) leave the
// registers to keep B's fragments of 64 r from block to block instead of 32.
// LONG: R over what is kept, B's fragments are loaded again for every block.
// 4096 x 4096 x 8192 with rank 32 (bf16), called in turn with the dense product of
// the same sizes: 208 to 218 us, 1.26 PFLOP/s and up; that one, which is the K loop,
// 189 to 194 (both are bound by the matrix unit under the chip's clock).
template <int DT, bool BKM, int BT, int TH, bool LONG>
__global__ __launch_bounds__(NT, BT == 128 ? 2 : 1) void lora_tile_kernel(LoraK a, int tiles_m, int tiles_n) {
    constexpr int BM = BT, BN = BT, TM = BM / 32, TN = BN / 32;
    constexpr int STAGE = (BM + BN) * KSTEP * 2;
    __shared__ __attribute__((aligned(1024))) char smem0[STAGE];
    __shared__ __attribute__((aligned(1024))) char smem1[STAGE];
    __shared__ int row_s[BM], ad_s[BM];
    __shared__ float undo_s[DT == 1 ? BM : 1];  // (of the first 64 r)
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int w = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    int tm, tn;
    grouped_order(w, tiles_m, tiles_n, 4, tm, tn);
    const int M = (int)a.M, N = (int)a.N, K = (int)a.K, R = a.R;
    const int m0 = tm * BM, n0 = tn * BN;
    for (int r = t; r < BM; r += NT) {
        const int p = m0 + r, m = p < M ? row_of(a, p) : -1, ad = m < 0 ? -1 : (int)row_adapter(a, m);
        row_s[r] = m;
        ad_s[r] = ad;
        if constexpr (DT == 1) undo_s[r] = ad < 0 || R == 0 ? 1.0f : row_undo(a, p, 0);
    }
    __syncthreads();
    GatherDma<BM> srcA;
    srcA.base = (const char*)a.X;
    srcA.K = K;
    srcA.lane = lane;
#pragma unroll
    for (int j = 0; j < GatherDma<BM>::PER_WAVE; ++j) {
        const int m = row_s[GatherDma<BM>::row_of(wave, j, lane)];
        srcA.roff[j] = m >= 0 ? (uint32_t)m * (uint32_t)K * 2u + (GatherDma<BM>::chunk(j, lane) << 4) : DMA_OOB;
    }
    DmaSrc<BN, BKM> srcB;
    srcB.init(a.W, BKM ? K : N, n0, N, K, lane);
    f32x4_t acc[TM][TN];
    const int nk = (K + KSTEP - 1) / KSTEP;
    if (n0 + BN <= N && K % KSTEP == 0)
        mainloop_dma16<BM, BN, DT, true, BKM, false>(acc, smem0, smem1, srcA, srcB, nk, lane, wm, wn, wave);
    else
        mainloop_dma16<BM, BN, DT, true, BKM, true>(acc, smem0, smem1, srcA, srcB, nk, lane, wm, wn, wave);

    // d = T B of block i of the wave (rows 16 i .. + 15) and TH column fragments
    // from jh on, in the accumulators' layout, one adapter of the block after
    // another.  Lane l: row l % 16, r = r0 + 8 (l / 16) .. + 7.  The accumulators
    // themselves are only read: an epilogue that multiplied into them made the
    // compiler spill them.
    const int i16 = lane & 15, q = (lane >> 4) * 8, row0 = wm * (BM / 2), col0 = wn * (BN / 2);
    const uint16_t* Bp = (const uint16_t*)a.B;
    constexpr int HS = TH == 8 ? 1 : 2;
    u32x4_t bf[LONG ? 1 : HS][TH];  // B's fragments
    int held = -1;
    // BKM = false: 32 r of 64 columns pass through LDS for the transposing read
    // (where no tile is staged, in the K loop's)
    __shared__ u32x4_t bt_s[BKM || BT == 128 ? 1 : 4 * 256];
    u32x4_t* bt = BT == 128 ? (u32x4_t*)smem0 + wave * 256 : bt_s + (BKM ? 0 : wave * 256);
    auto load_b = [&](u32x4_t (&f)[TH], int g, int r0, int jh) {
        const int c = n0 + col0 + 16 * jh;
        if constexpr (BKM) {
            const int n = max(0, min(8, R - r0 - q));
#pragma unroll
            for (int j = 0; j < TH; ++j)
                f[j] = load16_first(Bp + ((int64_t)g * N + min(c + 16 * j + i16, N - 1)) * R + r0 + q, n);
        } else {
#pragma unroll
            for (int h = 0; h < TH; h += 4) {
                const uint16_t* p = Bp + ((int64_t)g * R + r0) * N + min(c + 16 * h + 8 * (lane & 7), N - 8);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = 8 * u + (lane >> 3);
                    f[h + u] = r0 + r < R ? load16(p + (int64_t)r * N) : u32x4_t{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int h = 0; h < TH; h += 4) {
#pragma unroll
                for (int u = 0; u < 4; ++u) bt[u * 64 + lane] = f[h + u];
                __builtin_amdgcn_wave_barrier();
                const char* l = (const char*)bt + (q + (i16 >> 2)) * 128 + 8 * (i16 & 3);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OMM_LDS(i16x4_t, l + 32 * j));
                    const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OMM_LDS(i16x4_t, l + 32 * j + 4 * 128));
                    const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
                    f[h + j] = u32x4_t{l2.x, l2.y, h2.x, h2.y};
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
    };
    const int rp = (R + 7) & ~7;
    const int64_t plane = a.M * rp;
    auto t_row = [&](int i) { return a.Tp + (int64_t)min(m0 + row0 + 16 * i + i16, M - 1) * rp + q; };
    auto load_t = [&](u32x4_t (&part)[kParts32], const uint16_t* tp, int r0) {
#pragma unroll
        for (int h = 0; h < kParts32; ++h)
            part[h] = r0 + q < rp ? *(const u32x4_t*)(tp + h * plane + r0) : u32x4_t{0, 0, 0, 0};
    };
    u32x4_t ahead[kParts32];  // the next block's first step of T
    load_t(ahead, t_row(0), 0);
    auto delta = [&](int i, int jh, f32x4_t (&d)[TH]) {
#pragma unroll
        for (int j = 0; j < TH; ++j) d[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        const int ad = ad_s[row0 + 16 * i + i16];
        const u32x4_t first[kParts32] = {ahead[0], ahead[1], ahead[2]};
        load_t(ahead, t_row(i + 1 < TM ? i + 1 : 0), 0);
        for (uint32_t todo = (uint32_t)__ballot(ad >= 0) & 0xffffu; todo;) {
            const int g = __builtin_amdgcn_readlane(ad, __ffs(todo) - 1);
            todo &= ~(uint32_t)__ballot(ad == g);
            f32x4_t v[TH] = {};
            const auto step = [&](const u32x4_t (&f)[TH], int r0) {
                u32x4_t part[kParts32] = {first[0], first[1], first[2]};
                if (r0) load_t(part, t_row(i), r0);
#pragma unroll
                for (int h = 0; h < kParts32; ++h)
#pragma unroll
                    for (int j = 0; j < TH; ++j) v[j] = mfma16x16x32<DT>(f[j], part[h], v[j]);
            };
            // adds the rows of this adapter; fp16: of 64 r, which have a scale of their own
            const auto add = [&](float undo) {
#pragma unroll
                for (int j = 0; j < TH; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[j][e] = ad == g ? fmaf(v[j][e], undo, d[j][e]) : d[j][e];
            };
            const float undo = DT == 1 ? undo_s[row0 + 16 * i + i16] : 1.0f;
            if constexpr (!LONG) {
                if (held != g) {
#pragma unroll
                    for (int h = 0; h < HS; ++h)
                        if (32 * h < R) load_b(bf[h], g, 32 * h, jh);
                    held = g;
                }
#pragma unroll
                for (int h = 0; h < HS; ++h)
                    if (32 * h < R) step(bf[h], 32 * h);
#pragma unroll
                for (int j = 0; j < TH; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[j][e] = ad == g ? (DT == 1 ? v[j][e] * undo : v[j][e]) : d[j][e];
            } else {
                for (int r0 = 0; r0 < R; r0 += 32) {
                    load_b(bf[0], g, r0, jh);
                    step(bf[0], r0);
                    if (DT == 1 && (r0 & 32) && r0 + 32 < R) {
                        add(r0 < 64 ? undo : row_undo(a, min(m0 + row0 + 16 * i + i16, M - 1), r0 / 64));
#pragma unroll
                        for (int j = 0; j < TH; ++j) v[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                }
                add(DT == 1 && R > 64 ? row_undo(a, min(m0 + row0 + 16 * i + i16, M - 1), (R - 1) / 64) : undo);
            }
        }
    };

    uint16_t* Y = (uint16_t*)a.Y;
    const uint16_t* bias = (const uint16_t*)a.bias;
    // whole tiles leave through LDS as whole row segments (16-byte chunk c of
    // row r in slot c ^ (r % 16)), others by 4 columns
    const bool staged = BT == 256 && n0 + BN <= N && N % 8 == 0 && ((uintptr_t)Y & 15) == 0;
    char* stage = (wave < 2 ? smem0 : smem1) + (wave & 1) * (STAGE / 2);
    __syncthreads();  // every wave is done reading the last stage
    static_for<0, TN / TH>([&](auto hc) {
        constexpr int jh = decltype(hc)::value * TH;
        held = -1;
        float cb[TH][4];
#pragma unroll
        for (int j = 0; j < TH; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + col0 + 16 * (jh + j) + 4 * (lane >> 4) + e;
                cb[j][e] = bias && n < N ? from_bits<DT>(bias[n]) : 0.0f;
            }
        static_for<0, TM>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            f32x4_t d[TH];
            delta(i, jh, d);
            const int m = row_s[row0 + 16 * i + i16];
#pragma unroll
            for (int j = 0; j < TH; ++j) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][jh + j][e] + d[j][e] + cb[j][e];
                const u32x2_t o = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
                const int h = lane >> 4, n = n0 + col0 + 16 * (jh + j) + 4 * h;
                if (staged) {
                    const int c = 2 * (jh + j) + (h >> 1);
                    *(u32x2_t*)(stage + (16 * i + i16) * 256 + ((c ^ i16) << 4) + ((h & 1) << 3)) = o;
                } else if (m >= 0 && n < N) {
                    uint16_t* y = Y + (int64_t)m * N + n;
                    if (n + 4 <= N) {
                        typedef u32x2_t u32x2_u2 __attribute__((aligned(2)));
                        *(u32x2_u2*)y = o;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < N) y[e] = to_bits<DT>(v[e]);
                    }
                }
            }
        });
    });
    if (!staged) return;
    uint16_t* yb = Y + n0 + col0 + 8 * (lane & 15);
#pragma unroll 8
    for (int k = 0; k < 4 * TM; ++k) {
        const int r = 4 * k + (lane >> 4), m = row_s[row0 + r];
        const u32x4_t d = *(const u32x4_t*)(stage + r * 256 + (((lane & 15) ^ (r % 16)) << 4));
        if (m >= 0) *(u32x4_t*)(yb + (int64_t)m * N) = d;
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int DT, int TRANS>
void shrink(const LoraK& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.M + 15) / 16), (unsigned)shrink_parts(a.R));
    switch (shrink_cols(a.R)) {
        case 16: return lora_shrink_rows_kernel<DT, TRANS, 1, 16><<<grid, 1024, 0, s>>>(a);
        case 32: return lora_shrink_rows_kernel<DT, TRANS, 2, 16><<<grid, 1024, 0, s>>>(a);
        default: return lora_shrink_rows_kernel<DT, TRANS, 4, 8><<<grid, 512, 0, s>>>(a);
    }
}

template <int DT, int TRANS>
void expand(const LoraK& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 127) / 128), (unsigned)((a.M + 63) / 64));
    lora_expand_kernel<DT, TRANS><<<grid, 256, 0, s>>>(a);
}

template <int DT, int TRANS>
hipError_t rows_run(const LoraK& a, hipStream_t s) {
    if (a.perm && a.R > 0 && a.G > 0)
        lora_sort_kernel<<<1, 64 * kSortWaves, kSortWaves * (a.G + 1) * sizeof(int), s>>>(a, (int)a.G + 1);
    if (a.R > 0 && a.G > 0) {
        if (DT < 2 && !TRANS && a.R < 8) {  // (no group of 8 columns of A)
            lora_shrink_any(a, DT, s);
            if constexpr (DT < 2) lora_split_kernel<DT><<<dim3((unsigned)((a.M + 255) / 256)), 256, 0, s>>>(a);
        } else {
            shrink<DT, TRANS>(a, s);
        }
    }
    if constexpr (DT < 2) {
        if (lora_tiles_ok(a, DT)) {
            const int64_t big = (a.M + 255) / 256 * ((a.N + 255) / 256);
            if (big >= 256) {
                const int tm = (int)((a.M + 255) / 256), tn = (int)((a.N + 255) / 256);
                log_choice("lora_matmul: 256x256 tiles over sorted rows");
                const dim3 grid((unsigned)(tm * tn));
                if (a.R <= 32) lora_tile_kernel<DT, TRANS != 0, 256, 8, false><<<grid, NT, 0, s>>>(a, tm, tn);
                else if (a.R <= 64) lora_tile_kernel<DT, TRANS != 0, 256, 4, false><<<grid, NT, 0, s>>>(a, tm, tn);
                else lora_tile_kernel<DT, TRANS != 0, 256, 4, true><<<grid, NT, 0, s>>>(a, tm, tn);
            } else {
                const int tm = (int)((a.M + 127) / 128), tn = (int)((a.N + 127) / 128);
                log_choice("lora_matmul: 128x128 tiles over sorted rows");
                const dim3 grid((unsigned)(tm * tn));
                if (a.R <= 64) lora_tile_kernel<DT, TRANS != 0, 128, 4, false><<<grid, NT, 0, s>>>(a, tm, tn);
                else lora_tile_kernel<DT, TRANS != 0, 128, 4, true><<<grid, NT, 0, s>>>(a, tm, tn);
            }
            return hipGetLastError();
        }
    }
    log_choice("lora_matmul: adapters into Y, then the dense product");
    expand<DT, TRANS>(a, s);
    hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : lora_add_dense(a, a.Y, DT, s);
}

}  // namespace

// 16-byte rows for the DMA, 32-bit byte offsets into X and a tile of W
bool lora_tiles_ok(const LoraK& a, int dt) {
    return dt < 2 && a.K % 8 == 0 && a.K > 0 && (a.trans || a.N % 8 == 0) &&
           (((uintptr_t)a.X | (uintptr_t)a.W) & 15) == 0 && a.M * a.K * 2 < (1LL << 31) &&
           256 * (a.trans ? a.K : a.N) * 2 < (1LL << 31);
}

// whole groups of 8 (columns of a fp32 group: 4), one adapter's matrices within
// 32-bit offsets
bool lora_rows_ok(int64_t K, int64_t N, int64_t R, int64_t G) {
    return K >= 8 && N >= 8 && K * R < (1LL << 30) && N * R < (1LL << 30) &&
           K < (1 << 30) && N < (1 << 30) && G < (1LL << 31) - 1;
}

// the order of the rows, the parts' factors, T or its parts, and T where it is split by a kernel of its own
size_t lora_rows_workspace_bytes(int64_t M, int64_t R) {
    const size_t whole = align256((size_t)M * R * 4), parts = align256((size_t)kParts32 * M * ((R + 7) / 8 * 8) * 2);
    return align256((size_t)M * 4) + align256((size_t)M * shrink_parts((int)R) * 4) +
           std::max(whole, parts + (R < 8 ? whole : 0));
}

hipError_t launch_lora_rows(LoraK a, int dt, void* ws, hipStream_t s) {
    char* w = (char*)ws;
    a.perm = a.G < 1024 ? (int32_t*)w : nullptr;  // (more adapters than the sort has counters for: rows as they come)
    w += align256((size_t)a.M * 4);
    a.undo = (float*)w;
    w += align256((size_t)a.M * shrink_parts(a.R) * 4);
    a.Tp = (uint16_t*)w;
    a.T = dt == 2 ? (float*)w : (float*)(w + align256((size_t)kParts32 * a.M * ((a.R + 7) / 8 * 8) * 2));
    if (a.R == 0 || a.G == 0) a.perm = nullptr;
    switch (dt * 2 + a.trans) {
        case 0: return rows_run<0, 0>(a, s);
        case 1: return rows_run<0, 1>(a, s);
        case 2: return rows_run<1, 0>(a, s);
        case 3: return rows_run<1, 1>(a, s);
        case 4: return rows_run<2, 0>(a, s);
        default: return rows_run<2, 1>(a, s);
    }
}

}  // namespace omm
