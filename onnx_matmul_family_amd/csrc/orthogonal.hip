// Orthogonalised update: Newton-Schulz steps on a matrix (or a batch of them).
//
//   X = G / |G| (Frobenius);  `steps` times:  A = X X^T,  B = a I + b A + c A^2,  X <- B X
//   (tall matrices: of G^T, the same odd polynomial of the singular values; X is
//   always as wide as tall or wider)
//
// The steps multiply what is small in X by up to 3.44 each, roundings included, so
// X, A and B are held to 22 bits: as two fp16 parts (value, and what its rounding
// leaves), scaled by 2^14.  Singular values stay below 1.21, those of B between 0.6
// and 3.4445, so no entry passes 3.4445 and the scaled ones stay below 56500 of
// fp16's 65504, while the second part's smallest step is 2^-38 of |G|: entries below 2^-17
// of it have fewer bits (1e-8: 12).  A product is hi hi + hi lo + lo hi on the matrix unit
// with fp32 sums (lo lo is 2^-22 of it).  Errors against 64 bits, of the largest value
// (512 x 1024 in fp32; in brackets the same steps as torch's fp32 products): noise 2.4e-6
// (6.9e-6), four directions 100 times above it 8.8e-6 (1.1e-5), a block of 1e-8 |G| beside
// one of |G| 5.5e-5 of its own (1.6e-7).
//
// Layout: a row's 32 columns are 128 bytes, 64 of the first parts and 64 of the
// second, so a 128-byte stage of the loop holds both parts of 32 k and gives three
// products: 2/3 of the fetches, LDS writes and LDS reads of three products one
// after the other.  A and B are symmetric: tiles on and above the diagonal are
// computed, and written twice, and read along their rows.  X is read along its rows
// for A and across them (transposing LDS reads) for B X.  Sides are padded with zeros
// to 32.
//
// What bounds it: large matrices, the matrix unit (4096 x 4096: B X 278 us, 1.48 PFLOP/s of
// fp16 products, the library's fp16 product of 8192^3 1.58; A 165 and B 171, 1.25 and
// 1.20 of the half that is needed, 1.39 and 1.34 with what diagonal tiles compute twice;
// the whole call 3.19 ms, its floor 2.61).
// Batches of middle ones, tiles that do not fill the last turn (16 of 1000 x 1024: 576
// tiles of A on 512 places).  Small ones, 17 launches of 5 to 10 us, half of it starting and
// storing, the rest one CU's fetches of its tiles (512 x 1024: 136 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.hpp"
#include "row_loop.hpp"
#include "stream_core.hpp"

namespace omm {

namespace {

using namespace core16;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 16384.0f, kUnscale = 1.0f / 16384.0f;
constexpr int kNormBlocks = 512;

// element (row, col) of a matrix of row length ld in two parts: its first part; the second is 32 further
__device__ __forceinline__ int64_t part_at(int64_t row, int col, int ld) {
    return row * (2 * (int64_t)ld) + (col >> 5) * 64 + (col & 31);
}

// value and rest as fp16, four at a time
__device__ __forceinline__ void split4(const float (&v)[4], u32x2_t& hi, u32x2_t& lo) {
    hi = u32x2_t{pack2<1>(v[0], v[1]), pack2<1>(v[2], v[3])};
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = v[e] - f16_bits_to_f32((uint16_t)(hi[e >> 1] >> (16 * (e & 1))));
    lo = u32x2_t{pack2<1>(r[0], r[1]), pack2<1>(r[2], r[3])};
}
__device__ __forceinline__ void join4(u32x2_t hi, u32x2_t lo, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = f16_bits_to_f32((uint16_t)(hi[e >> 1] >> (16 * (e & 1)))) +
               f16_bits_to_f32((uint16_t)(lo[e >> 1] >> (16 * (e & 1))));
}
// 4 x 4 16-bit values over four neighbouring lanes, transposed: a lane's four
// columns of its row become four rows of column lane % 4.
template <int PERM>
__device__ __forceinline__ u32x2_t quad(u32x2_t v) {
    return u32x2_t{(uint32_t)__builtin_amdgcn_mov_dpp((int)v.x, PERM, 0xf, 0xf, true),
                   (uint32_t)__builtin_amdgcn_mov_dpp((int)v.y, PERM, 0xf, 0xf, true)};
}
__device__ __forceinline__ u32x2_t transpose4(u32x2_t v, int lane) {
    const u32x2_t o = quad<0xb1>(v);  // the lane's neighbour (1, 0, 3, 2)
    const bool odd = lane & 1;
    u32x2_t p;  // even: columns 0 and 2 of two rows, odd: columns 1 and 3
#pragma unroll
    for (int i = 0; i < 2; ++i)
        p[i] = odd ? __builtin_amdgcn_perm(v[i], o[i], 0x07060302u) : __builtin_amdgcn_perm(o[i], v[i], 0x05040100u);
    const u32x2_t r = quad<0x4e>(p);  // the lane two further (2, 3, 0, 1)
    return lane & 2 ? u32x2_t{r.y, p.y} : u32x2_t{p.x, r.x};
}

// ------------------------------------------------------------------ G / |G|
// sum of the squares of one matrix, in 64 bits: parts[z][block]; and the join's counters are cleared
template <int DT>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const void* G, int64_t mn, double* parts, uint32_t* joined, int njoined) {
    typedef typename elem_of<DT>::type E;
    constexpr int V = kVec<DT>;
    __shared__ double red[4];
    const E* g = (const E*)G + (int64_t)blockIdx.y * mn;
    if (blockIdx.x == 0 && blockIdx.y == 0 && (int)threadIdx.x < njoined) joined[threadIdx.x] = 0;
    double s = 0.0;
    for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; e < mn; e += (int64_t)gridDim.x * 256 * V) {
        float f[V];
        unpack16<DT>(load16_first(g + e, (int)min((int64_t)V, mn - e)), f);
#pragma unroll
        for (int i = 0; i < V; ++i) s += (double)f[i] * (double)f[i];
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) parts[(int64_t)blockIdx.y * kNormBlocks + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// 64 x 64 of X = G / |G| in two parts; of G^T where G is tall.  All NaN if G holds a
// NaN or an infinity.  rows, cols: X's padded sides.
template <int DT>
__global__ __launch_bounds__(256) void ortho_split_kernel(const void* G, int m, int n, int tall, int rows, int cols,
                                                          const double* parts, int nparts, uint16_t* X) {
    typedef typename elem_of<DT>::type E;
    __shared__ double red[4];
    __shared__ float tile[64][65];
    const int64_t z = blockIdx.y;
    const int t = threadIdx.x;
    // the block's corner in X and in G
    const int tc = (cols + 63) / 64, r0 = (int)(blockIdx.x / tc) * 64, c0 = (int)(blockIdx.x % tc) * 64;
    const int gr = tall ? c0 : r0, gc = tall ? r0 : c0;
    const E* g = (const E*)G + z * (int64_t)m * n;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = gr + 4 * i + (t >> 6), c = gc + (t & 63);
        v[i] = r < m && c < n ? elem_f32<DT>(g[(int64_t)r * n + c]) : 0.0f;
    }
    double s = 0.0;
    for (int i = t; i < nparts; i += 256) s += parts[z * kNormBlocks + i];
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, 64);
    if ((t & 63) == 0) red[t >> 6] = s;
    __syncthreads();
    s = (red[0] + red[1]) + (red[2] + red[3]);
    const double factor = s == 0.0 ? 0.0 : s < __builtin_inf() ? (double)kScale / sqrt(s) : __builtin_nan("");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = (float)((double)v[i] * factor);
        const int a = 4 * i + (t >> 6), b = t & 63;
        const bool in = gr + a < m && gc + b < n;  // (the padding is 0 beside NaN too)
        (tall ? tile[b][a] : tile[a][b]) = in ? x : 0.0f;
    }
    __syncthreads();
    X += z * 2 * rows * cols;
    // 16 lanes a row of 4 values each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = 16 * i + (t >> 4), b = 4 * (t & 15);
        if (r0 + a >= rows || c0 + b >= cols) continue;
        float w[4];
        u32x2_t hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = tile[a][b + e];
        split4(w, hi, lo);
        uint16_t* d = X + part_at(r0 + a, c0 + b, cols);
        *(u32x2_t*)d = hi;
        *(u32x2_t*)(d + 32) = lo;
    }
}

// ------------------------------------------------------------------ products
// R columns of an operand (K, cols) whose rows run across the contraction: 32 rows of
// 4 R bytes a stage, 32-byte granules permuted as in the MN-major tiles of
// device_common.hpp.  Columns past the last read on into the next row (their results
// are not stored); past the operand's end, zeros.
template <int R>
struct ColSrc {
    static constexpr int PER_WAVE = R / 32, ROWB = 4 * R;
    const char* base;
    int64_t step, bytes;  // of a stage, from the tile's first column to the operand's end
    uint32_t off[PER_WAVE];
    __device__ __forceinline__ void init(const uint16_t* p, int cols, int K, int col0, int wave, int lane) {
        const uint32_t ldb = (uint32_t)cols * 4u;
        base = (const char*)p + (int64_t)col0 * 4;
        step = 32 * (int64_t)ldb;
        bytes = (int64_t)K * ldb - (int64_t)col0 * 4;
#pragma unroll
        for (int j = 0; j < PER_WAVE; ++j) {
            const int at = (wave * PER_WAVE + j) * 1024 + lane * 16, k = at / ROWB, c = at % ROWB / 16;
            off[j] = (uint32_t)k * ldb + (uint32_t)(2 * ((c >> 1) ^ mswz16(k)) + (c & 1)) * 16u;
        }
    }
    __device__ __forceinline__ i32x4_t rsrc(int kt, int nk) const {
        i32x4_t r = make_rsrc(base + (kt < nk ? kt * step : 0));
        r.z = __builtin_amdgcn_readfirstlane(kt < nk ? (int)min(bytes - kt * step, (int64_t)0x7fffffff) : 0);
        return r;
    }
    __device__ __forceinline__ void one(const i32x4_t& r, uint32_t lds, int, int wave, int j) const {
        dma16u(r, lds + (wave * PER_WAVE + j) * 1024, off[j]);
    }
    // fragment of columns [col, col + 16), part p
    __device__ __forceinline__ static u32x4_t read(const char* lds, int col, int p, int lane) {
        const int i = lane & 15, k = 8 * (lane >> 4) + (i >> 2), c = col + 4 * (i & 3);
        const int byte = (c >> 5) * 128 + p * 64 + (c & 31) * 2;
        const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OMM_LDS(i16x4_t, lds + mmaj16_off<ROWB>(k, byte)));
        const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OMM_LDS(i16x4_t, lds + mmaj16_off<ROWB>(k + 4, byte)));
        const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
        return u32x4_t{l2.x, l2.y, h2.x, h2.y};
    }
};

// acc = sum over nk stages of hi hi + hi lo + lo hi.  NB stages in LDS, all but
// the current one on their way.  A stage's three phases: hi hi (while the columns'
// second parts are read), hi lo (the rows'), the barrier that retires the stage's
// buffer and publishes the next, lo hi (the next stage's first parts, and the DMA of
// stage kt + NB into the retired buffer).  P: which of fb holds the first parts.
// SB: RowSrc or ColSrc.  The loop begins with stage `first` and ends with the one before it.
template <int BT, int NB, class SB>
struct Loop {
    static constexpr int TM = BT / 32, NM = TM * TM, OPB = BT * 128, STAGE = 2 * OPB, LA = RowSrc<BT>::PER_WAVE;
    f32x4_t (&acc)[TM][TM];
    char* smem;
    const RowSrc<BT>& sa;
    const SB& sb;
    int nk, first, lane, wave, rowa, rowb;
    u32x4_t fa[2][TM], fb[2][TM];

    __device__ __forceinline__ char* at(int kt) const { return smem + (kt % NB) * STAGE; }
    template <int p>
    __device__ __forceinline__ u32x4_t reada(const char* st, int i) const {
        return read_frag16<BT, true>(st, rowa + 16 * i, p, lane);
    }
    template <int p>
    __device__ __forceinline__ u32x4_t readb(const char* st, int i) const {
        if constexpr (std::is_same<SB, RowSrc<BT>>::value) return read_frag16<BT, true>(st + OPB, rowb + 16 * i, p, lane);
        else return SB::read(st + OPB, rowb + 16 * i, p, lane);
    }
    __device__ __forceinline__ int turned(int kt) const { return kt < nk ? (kt + first < nk ? kt + first : kt + first - nk) : nk; }
    __device__ __forceinline__ void issue(int kt) const {
        const i32x4_t ra = sa.rsrc(turned(kt), nk), rb = sb.rsrc(turned(kt), nk);
        const uint32_t l = lds_addr(at(kt));
#pragma unroll
        for (int j = 0; j < LA; ++j) sa.one(ra, l, kt, wave, j);
#pragma unroll
        for (int j = 0; j < LA; ++j) sb.one(rb, l + OPB, kt, wave, j);
    }
    template <int P, bool Z>
    __device__ __forceinline__ void stage(int kt) {
        const char *st = at(kt), *nx = at(kt + 1);
        phase<1, TM, TM, Z>(acc, fa[0], fb[P], [&](auto xc) {
            spread<NM, TM, decltype(xc)::value>([&](auto i) { fb[P ^ 1][i] = readb<1>(st, i); });
        });
        phase<1, TM, TM, false>(acc, fa[0], fb[P ^ 1], [&](auto xc) {
            spread<NM, TM, decltype(xc)::value>([&](auto i) { fa[1][i] = reada<1>(st, i); });
        });
        wait_vm<(NB - 2) * 2 * LA>();  // this wave's DMA of stage kt + 1 has landed
        __syncthreads();               // ... every wave's; and every read of stage kt is done
        fence_sched();
        const int next = turned(kt + NB);
        const i32x4_t ra = sa.rsrc(next, nk), rb = sb.rsrc(next, nk);
        const uint32_t l = lds_addr(st);
        phase<1, TM, TM, false>(acc, fa[1], fb[P], [&](auto xc) {
            constexpr int x = decltype(xc)::value;
            spread<NM, 2 * LA, x>([&](auto d) {
                if constexpr (decltype(d)::value < LA) sa.one(ra, l, kt + NB, wave, d);
                else sb.one(rb, l + OPB, kt + NB, wave, d - LA);
            });
            spread<NM, 2 * TM, x>([&](auto r) {
                constexpr int i = decltype(r)::value / 2;
                if constexpr (decltype(r)::value % 2 == 0) fb[P ^ 1][i] = readb<0>(nx, i);
                else fa[0][i] = reada<0>(nx, i);
            });
        });
    }
    __device__ __forceinline__ void run() {
        for (int kt = 0; kt < NB; ++kt) issue(kt);
        wait_vm<(NB - 1) * 2 * LA>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            fa[0][i] = reada<0>(smem, i);
            fb[0][i] = readb<0>(smem, i);
        }
        stage<0, true>(0);
        int kt = 1;
        for (; kt + 2 <= nk; kt += 2) {
            stage<1, false>(kt);
            stage<0, false>(kt + 1);
        }
        if (kt < nk) stage<1, false>(kt);
        wait_vm<0>();
        acc_fence(acc);
    }
};

// The same for 32 x 32 tiles, which are for matrices that make few others: each of 8
// waves takes every 8th stage for itself, NB of them on their way in LDS of its own
// (no barrier), and the waves' sums join in LDS, in their order.  The first wave
// returns with the tile.
struct SmallLoop {
    static constexpr int NB = 2, WAVES = 8, OPB = 32 * 128, STAGE = 2 * OPB, LDS = WAVES * NB * STAGE;
    typedef RowSrc<32, false, 1> S;
    static __device__ __forceinline__ void run(f32x4_t (&acc)[2][2], char* smem, const S& sa, const S& sb, int nk, int lane,
                                               int wave) {
        char* own = smem + wave * (NB * STAGE);
        const auto issue = [&](int i) {
            const int kt = min(i * WAVES + wave, nk);
            const i32x4_t ra = sa.rsrc(kt, nk), rb = sb.rsrc(kt, nk);
            const uint32_t l = lds_addr(own + (i % NB) * STAGE);
#pragma unroll
            for (int j = 0; j < 4; ++j) sa.one(ra, l, kt, 0, j);
#pragma unroll
            for (int j = 0; j < 4; ++j) sb.one(rb, l + OPB, kt, 0, j);
        };
        const int n = (nk + WAVES - 1) / WAVES;
#pragma unroll
        for (int i = 0; i < NB; ++i) issue(i);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < n; ++i) {
            wait_vm<(NB - 1) * 8>();
            asm volatile("" ::: "memory");
            const char* st = own + (i % NB) * STAGE;
            u32x4_t fa[2][2], fb[2][2];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    fa[p][h] = read_frag16<32, true>(st, 16 * h, p, lane);
                    fb[p][h] = read_frag16<32, true>(st + OPB, 16 * h, p, lane);
                }
            // (the values are here before the buffer is filled again)
            asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(fa[0][0]), "+v"(fa[0][1]), "+v"(fa[1][0]), "+v"(fa[1][1]),
                         "+v"(fb[0][0]), "+v"(fb[0][1]), "+v"(fb[1][0]), "+v"(fb[1][1])::"memory");
            issue(i + NB);
#pragma unroll
            for (int q = 0; q < 3; ++q)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    acc[x >> 1][x & 1] = mfma16x16x32<1>(fb[q == 1][x & 1], fa[q == 2][x >> 1], acc[x >> 1][x & 1]);
        }
        wait_vm<0>();
        __syncthreads();
        f32x4_t* red = (f32x4_t*)smem;
#pragma unroll
        for (int x = 0; x < 4; ++x) red[(wave * 4 + x) * 64 + lane] = acc[x >> 1][x & 1];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int w = 1; w < WAVES; ++w) acc[x >> 1][x & 1] += red[(w * 4 + x) * 64 + lane];
    }
};

enum OrthoOp { kGram, kPoly, kUpdate };

struct OrthoK {
    const uint16_t* A;  // (rows, K): rows of the result
    const uint16_t* B;  // (cols, K): its columns; kUpdate: (K, cols)
    uint16_t* D;        // (rows, cols), the result
    void* out;          // or, of the last step, T
    int rows, cols, K;  // padded
    int m, n;           // of out: (rows, cols) without padding, or (cols, rows) of a tall G
    int tall;
    int tiles;          // of one matrix
    // kGram of few tiles and a long contraction: `split` workgroups a tile, whose sums meet here
    int split;
    uint64_t* sums;     // [tile][split][wave][2 TM TM][64], pairs of fp32
    uint32_t* joined;   // [tile]: workgroups whose sums are there; 0 before and after a launch
};
constexpr int kSplitPlaces = 256;  // workgroups of a launch that is split

// DT: 3 = in two parts, else T of the last step's result
// H: side of a wave's block
template <int OP, int DT, int BT, int NB>
__global__ __launch_bounds__(BT == 32 ? 512 : NT, NB * BT * 256 <= 80 * 1024 ? 2 : 1) void ortho_kernel(OrthoK a) {
    constexpr bool SYM = OP != kUpdate, LAST = DT < 3, SMALL = BT == 32;
    constexpr int H = SMALL ? 32 : BT / 2, TM = H / 16;
    __shared__ __attribute__((aligned(1024))) char smem[SMALL ? SmallLoop::LDS : NB * BT * 256];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = SMALL ? 0 : wave >> 1, wn = SMALL ? 0 : wave & 1;
    constexpr bool SPLIT = OP == kGram && BT <= 64;
    const int wall = xcd_remap((int)blockIdx.x, (int)gridDim.x), part = SPLIT ? wall % a.split : 0;
    const int w = SPLIT ? wall / a.split : wall;
    const int z = w / a.tiles;
    int tm, tn, i = w - z * a.tiles;
    const int T = (a.rows + BT - 1) / BT;
    if constexpr (SYM) {
        // i-th of the tiles tn >= tm, row by row
        tm = 0;
        while (i >= T - tm) i -= T - tm++;
        tn = tm + i;
    } else {
        grouped_order(i, T, (a.cols + BT - 1) / BT, 4, tm, tn);
    }
    const int m0 = tm * BT, n0 = tn * BT;
    // 32 rows of the wave's columns at a time pass through LDS, so that A is read and
    // the results are written by whole rows of 16 bytes a lane (8 bytes a lane straight
    // from the accumulators' layout: 45 us a 256 x 256 tile on an idle chip).  All of it
    // is the wave's own: no barrier.  Rows are of W bytes; of the transposed result 32
    // rows are 128 bytes of each column.  Small tiles, where the registers are there,
    // ask for A's before the loop.
    constexpr bool AHEAD = BT <= 128;
    constexpr int W = H * 4, CPR = W / 16, NCH = 32 * CPR / 64;
    const int64_t size = (int64_t)z * 2 * a.rows * a.cols;
    const uint16_t* C = a.A + size;  // kPoly: A itself
    uint16_t* D = a.D + size;
    char *direct = smem + wave * (32 * W + H * 128), *across = direct + 32 * W;
    const int wr = m0 + wm * H, wc = n0 + wn * H;
    // 16-byte piece of 32 columns' 128 bytes, by row: neighbouring rows in other banks
    const auto slot = [](int row, int piece) { return (piece ^ (row & 7)) << 4; };
    u32x4_t cr[OP == kPoly ? NCH : 1];
    const auto load_c = [&](int r0) {
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
            const int row = (q * 64 + lane) / CPR, ch = (q * 64 + lane) % CPR;
            cr[q] = r0 + row < a.rows && wc + ch / 8 * 32 < a.cols
                        ? *(const u32x4_t*)(C + part_at(r0 + row, wc, a.cols) + ch * 8) : u32x4_t{0, 0, 0, 0};
        }
    };
    if constexpr (OP == kPoly && AHEAD) load_c(wr);
    f32x4_t acc[TM][TM];
    const int from = SPLIT ? part * (a.K / 32) / a.split : 0;  // stages of this part
    const int nk = (SPLIT ? (part + 1) * (a.K / 32) / a.split : a.K / 32) - from;
    const uint16_t *A = a.A + (int64_t)z * 2 * a.rows * a.K, *B = a.B + (int64_t)z * 2 * a.cols * a.K;
    if constexpr (SMALL) {
        SmallLoop::S sa, sb;
        sa.init(A, a.K * 4, a.K * 4, m0, a.rows, lane);
        sb.init(B, a.K * 4, a.K * 4, n0, a.cols, lane);
        if constexpr (SPLIT) {
            sa.skip(from);
            sb.skip(from);
        }
        SmallLoop::run(acc, smem, sa, sb, nk, lane, wave);
    } else {
        typedef typename std::conditional<SYM, RowSrc<BT>, ColSrc<BT>>::type SB;
        RowSrc<BT> sa;
        SB sb;
        sa.init(A, a.K * 4, a.K * 4, m0, a.rows, lane);
        if constexpr (SYM) sb.init(B, a.K * 4, a.K * 4, n0, a.cols, lane);
        else sb.init(B, a.cols, a.K, n0, wave, lane);
        if constexpr (SPLIT) {
            sa.skip(from);
            sb.skip(from);
        }
        // B X: a x, the largest part of a result in the first steps, comes with the stages
        // of the diagonal; as the last ones, so that the other terms are summed by themselves
        // and not on top of it (1000 x 1000 in fp32: 2.0e-6 -> 1.7e-6 off)
        const int first = SYM ? 0 : min(m0 + BT, a.K) / 32 % nk;
        Loop<BT, NB, SB> loop{acc, smem, sa, sb, nk, first, lane, wave, wm * H, wn * H};
        loop.run();
    }

    __syncthreads();  // every wave is done with the last stage
    if constexpr (SPLIT) {
        // the last of a tile's workgroups to be here sums what all of them left, in their order
        if (a.split > 1) {
            constexpr int WAVES = SMALL ? 1 : 4, N = 2 * TM * TM;  // pairs of a lane
            uint64_t* mine = a.sums + ((int64_t)w * a.split * WAVES + wave) * (N * 64) + lane;
            constexpr int64_t PART = WAVES * N * 64;
            if (wave < WAVES) {
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const f32x4_t& v = acc[x / 2 / TM][x / 2 % TM];
                    const float pair[2] = {v[x % 2 * 2], v[x % 2 * 2 + 1]};
                    __hip_atomic_store(mine + part * PART + x * 64, __builtin_bit_cast(uint64_t, pair), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
                }
            }
            if (!part_last(a.joined + w, a.split, t)) return;
            if (wave < WAVES) {
                float sum[2 * N] = {};
#pragma unroll 2
                for (int p = 0; p < a.split; ++p) {
                    uint64_t u[N];
#pragma unroll
                    for (int x = 0; x < N; ++x)
                        u[x] = __hip_atomic_load(mine + p * PART + x * 64, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        sum[2 * x] += __uint_as_float((uint32_t)u[x]);
                        sum[2 * x + 1] += __uint_as_float((uint32_t)(u[x] >> 32));
                    }
                }
#pragma unroll
                for (int x = 0; x < 2 * N; ++x) acc[x / 4 / TM][x / 4 % TM][x % 4] = sum[x];
            }
            if (t == 0) __hip_atomic_store(a.joined + w, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (SMALL && wave) return;
    if constexpr (OP == kPoly && !AHEAD) load_c(wr);
#pragma unroll
    for (int h = 0; h < TM / 2; ++h) {
        const int r0 = wr + 32 * h;
        if (r0 >= a.rows) break;
        if constexpr (OP == kPoly) {
#pragma unroll
            for (int q = 0; q < NCH; ++q) {
                const int row = (q * 64 + lane) / CPR, ch = (q * 64 + lane) % CPR;
                *(u32x4_t*)(direct + row * W + (ch >> 3) * 128 + slot(row, ch & 7)) = cr[q];
            }
            if (h + 1 < TM / 2) load_c(r0 + 32);
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int ii = 0; ii < 2; ++ii) {
            const int i = 2 * h + ii, row = 16 * ii + (lane & 15), g = lane >> 4;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                // columns 16 j + 4 g .. + 3: half of piece (j & 1) * 2 + g / 2, and of that + 4
                const int pc = (j & 1) * 2 + (g >> 1);
                char* at = direct + row * W + (j >> 1) * 128 + (g & 1) * 8;
                u32x2_t *ph = (u32x2_t*)(at + slot(row, pc)), *pl = (u32x2_t*)(at + slot(row, pc + 4));
                const int r = r0 + row, c = wc + 16 * j + 4 * g;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * kUnscale;
                if constexpr (OP == kPoly) {
                    float x[4];
                    join4(*ph, *pl, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = (r == c + e ? kA * kScale : 0.0f) + (kB * x[e] + kC * v[e]);
                }
                if constexpr (LAST) {
                    // of T: 32 rows of H columns, or of a tall G H rows of 32
                    typedef typename elem_of<LAST ? DT : 2>::type E;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int col = 16 * j + 4 * g + e;
                        ((E*)direct)[a.tall ? col * (32 + kVec<DT>) + row : row * (H + kVec<DT>) + col] =
                            f32_elem<LAST ? DT : 2>(v[e] * kUnscale);
                    }
                } else {
                    u32x2_t hi, lo;
                    split4(v, hi, lo);
                    *ph = hi;
                    *pl = lo;
                    if (SYM && tm != tn) {
                        const int c = 16 * j + 4 * g + (lane & 3), pr = 2 * ii + ((lane & 15) >> 3);
                        char* to = across + c * 128 + ((lane >> 2) & 1) * 8;
                        *(u32x2_t*)(to + slot(c, pr)) = transpose4(hi, lane);
                        *(u32x2_t*)(to + slot(c, pr + 4)) = transpose4(lo, lane);
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (LAST) {
            const auto rows_out = [&](auto len, int row0, int col0) {
                typedef typename elem_of<LAST ? DT : 2>::type E;
                typedef typename std::conditional<DT == 2, u32x4_u4, u32x4_u2>::type u32x4_e;
                constexpr int L = decltype(len)::value, V = kVec<DT>, PER = L / V;
                E* out = (E*)a.out + (int64_t)z * a.m * a.n;
#pragma unroll
                for (int q = 0; q < 32 * H / V / 64; ++q) {
                    const int row = (q * 64 + lane) / PER, ch = (q * 64 + lane) % PER * V;
                    const E* from = (const E*)direct + row * (L + V) + ch;
                    const u32x4_t d = *(const u32x4_t*)from;
                    if (row0 + row >= a.m) continue;
                    E* to = out + (int64_t)(row0 + row) * a.n + col0 + ch;
                    if (col0 + ch + V <= a.n) {
                        *(u32x4_e*)to = d;
                    } else {
                        for (int e = 0; col0 + ch + e < a.n; ++e) to[e] = from[e];
                    }
                }
            };
            if (a.tall) rows_out(std::integral_constant<int, 32>{}, wc, r0);
            else rows_out(std::integral_constant<int, H>{}, r0, wc);
            __builtin_amdgcn_wave_barrier();
        } else {
#pragma unroll
            for (int q = 0; q < NCH; ++q) {
                const int row = (q * 64 + lane) / CPR, ch = (q * 64 + lane) % CPR;
                const u32x4_t d = *(const u32x4_t*)(direct + row * W + (ch >> 3) * 128 + slot(row, ch & 7));
                if (r0 + row < a.rows && wc + ch / 8 * 32 < a.cols)
                    *(u32x4_t*)(D + part_at(r0 + row, wc, a.cols) + ch * 8) = d;
            }
            if (SYM && tm != tn) {
#pragma unroll
                for (int q = 0; q < H / 8; ++q) {
                    const int c = 8 * q + (lane >> 3), ch = lane & 7;
                    const u32x4_t d = *(const u32x4_t*)(across + c * 128 + slot(c, ch));
                    if (wc + c < a.cols) *(u32x4_t*)(D + part_at(wc + c, r0, a.rows) + ch * 8) = d;
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t padded(int64_t n) { return (n + 31) / 32 * 32; }

// A and B, 4096 x 4096 (128 stages): 328 / 219 / 175 / 231 us with tiles of 64 / 128 / 192 / 256; 512 x 1024:
// 11.4 / 25 / 42 / 66; 16 of 1000 x 1024: 84 / 69 / 98 / 88.  B X: 463 / 329 / 378 / 284; 9.0 / 15.4 /
// 26 / 37; 160 / 100 / 152 / 91.
constexpr TileTimes kSymTiles[] = {{32, 256, 3.4, 0.12, 0.2, 0.2}, {64, 512, 3.4, 0.25, 0.3, 0.63},
                                   {128, 512, 11, 0.43, 0.6, 1.29}, {192, 256, 26, 0.5, 1.17, 1.17},
                                   {256, 256, 34, 1.0, 1.93, 1.93}};
constexpr TileTimes kUpdateTiles[] = {{64, 512, 4, 0.3, 0.35, 0.65}, {128, 512, 8.5, 0.43, 0.6, 1.3},
                                      {192, 256, 18, 0.5, 1.3, 1.3}, {256, 256, 21, 1.0, 2.05, 2.05}};

int64_t tiles_of(const OrthoK& k, bool sym, int bt) {
    const int64_t tm = (k.rows + bt - 1) / bt, tn = (k.cols + bt - 1) / bt;
    return sym ? tm * (tm + 1) / 2 : tm * tn;
}

// A = X X^T (p x p, contraction q) of tiles that leave CUs without one: by how many
// workgroups a tile's contraction is split, and the tile.  (The whole call, us, with one
// workgroup a tile and split: 64 x 2496 108 and 98, 96 x 4096 133 and 116, 384 x 3840 180 and
// 166, 18 of 3200 x 192 327 and 290; the parts pass the L2, as a fence for every workgroup's
// stores made the last 420.)
struct GramPlan {
    int bt, split;
    int64_t tiles;  // of the batch
    size_t sums_bytes() const { return split > 1 ? (size_t)tiles * split * bt * bt * 4 : 0; }
};
GramPlan gram_plan(int64_t Z, int64_t p, int64_t q) {
    constexpr double kJoin = 5.0;  // us, as measured (3: 512 x 1472 140 -> 142)
    OrthoK k = {};
    k.rows = k.cols = (int)p;
    const double stages = (double)(q / 32);
    GramPlan best = {};
    double least = 0.0;
    for (const TileTimes& t : kSymTiles) {
        const int64_t n = Z * tiles_of(k, true, t.bt);
        for (int split = 1; split <= 16; split *= 2) {
            if (split > 1 && (t.bt > 64 || n * split > kSplitPlaces || stages < 8 * split)) break;
            const double time = tile_time(t, n * split, stages / split) + (split > 1 ? kJoin : 0.0);
            if (!best.bt || time < least) {
                best = {t.bt, split, n};
                least = time;
            }
        }
    }
    return best;
}

template <int OP, int DT>
void product(OrthoK k, int64_t Z, hipStream_t s) {
    const auto count = [&](int bt) { return Z * tiles_of(k, OP != kUpdate, bt); };
    int bt;
    k.split = 1;
    if constexpr (OP == kGram) {
        const GramPlan plan = gram_plan(Z, k.rows, k.K);
        bt = plan.bt;
        k.split = plan.split;
    } else {
        bt = OP == kUpdate ? pick_tile(kUpdateTiles, k.K / 32, count) : pick_tile(kSymTiles, k.K / 32, count);
    }
    log_choice("orthogonalize: %d x %d x %d, tiles of %d, %d workgroups each", k.rows, k.cols, k.K, bt, k.split);
    k.tiles = (int)tiles_of(k, OP != kUpdate, bt);
    const unsigned grid = (unsigned)(k.tiles * Z * k.split);
    if (bt == 32) {
        if constexpr (OP != kUpdate) ortho_kernel<OP, DT, 32, 2><<<grid, 512, 0, s>>>(k);
    } else if (bt == 64) ortho_kernel<OP, DT, 64, 4><<<grid, NT, 0, s>>>(k);
    else if (bt == 128) ortho_kernel<OP, DT, 128, 2><<<grid, NT, 0, s>>>(k);
    else if (bt == 192) ortho_kernel<OP, DT, 192, 3><<<grid, NT, 0, s>>>(k);
    else ortho_kernel<OP, DT, 256, 2><<<grid, NT, 0, s>>>(k);
}

template <int DT>
hipError_t ortho_run(const OrthoArgs& o, void* ws, hipStream_t s) {
    const bool tall = o.m > o.n;
    const int64_t Z = o.batch, mn = o.m * o.n, p = padded(std::min(o.m, o.n)), q = padded(std::max(o.m, o.n));
    char* w = (char*)ws;
    double* parts = (double*)w;
    w += align256((size_t)Z * kNormBlocks * 8);
    uint16_t* X[2];
    for (auto& x : X) {
        x = (uint16_t*)w;
        w += align256((size_t)Z * 4 * p * q);
    }
    uint16_t* A = (uint16_t*)w;
    uint16_t* B = (uint16_t*)(w + align256((size_t)Z * 4 * p * p));
    w += 2 * align256((size_t)Z * 4 * p * p);
    const GramPlan plan = gram_plan(Z, p, q);
    OrthoK k;
    k.joined = (uint32_t*)w;
    k.sums = (uint64_t*)(w + kSplitPlaces * 4);
    const int nparts = (int)std::min<int64_t>(kNormBlocks, (mn + 8191) / 8192);
    ortho_norm_kernel<DT><<<dim3(nparts, (unsigned)Z), 256, 0, s>>>(o.G, mn, parts, k.joined,
                                                                    plan.split > 1 ? (int)plan.tiles : 0);
    const int64_t tiles = ((p + 63) / 64) * ((q + 63) / 64);
    ortho_split_kernel<DT><<<dim3((unsigned)tiles, (unsigned)Z), 256, 0, s>>>(
        o.G, (int)o.m, (int)o.n, tall, (int)p, (int)q, parts, nparts, X[0]);
    k.m = (int)o.m;
    k.n = (int)o.n;
    k.tall = tall;
    k.out = o.out;
    for (int step = 0; step < o.steps; ++step) {
        const int x = step & 1;
        k.rows = k.cols = (int)p;
        k.K = (int)q;
        k.A = k.B = X[x];
        k.D = A;
        product<kGram, 3>(k, Z, s);
        k.K = (int)p;
        k.A = k.B = A;
        k.D = B;
        product<kPoly, 3>(k, Z, s);
        k.cols = (int)q;
        k.A = B;
        k.B = X[x];
        k.D = X[x ^ 1];
        if (step + 1 == o.steps) product<kUpdate, DT>(k, Z, s);
        else product<kUpdate, 3>(k, Z, s);
    }
    return hipGetLastError();
}

}  // namespace

size_t orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n) {
    const int64_t mp = padded(m), np = padded(n), p = mp < np ? mp : np;
    const size_t sums = gram_plan(batch, p, mp < np ? np : mp).sums_bytes();
    return (sums ? kSplitPlaces * 4 + sums : 0) + align256((size_t)batch * kNormBlocks * 8) + 2 * align256((size_t)batch * 4 * mp * np) +
           2 * align256((size_t)batch * 4 * p * p);
}

hipError_t launch_orthogonalize(const OrthoArgs& a, int dt, void* ws, hipStream_t s) {
    return dt == 0 ? ortho_run<0>(a, ws, s) : dt == 1 ? ortho_run<1>(a, ws, s) : ortho_run<2>(a, ws, s);
}

}  // namespace omm
