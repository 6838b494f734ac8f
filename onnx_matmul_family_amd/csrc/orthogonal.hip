// Orthogonalised update: Newton-Schulz steps on a matrix (or a batch of them).
//
//   X = G / |G| (Frobenius);  `steps` times:  A = X X^T,  X <- a X + (b A + c A^2) X
//   (tall matrices: of G^T, the same odd polynomial of the singular values; X is
//   always as wide as tall or wider)
//
// The steps multiply what is small in X by up to 3.44 each, roundings included, so
// X, A and B = b A + c A^2 are held to 22 bits: as two fp16 parts (value, and what
// its rounding leaves), scaled by 2^14.  Singular values stay below 1.21, so no
// entry of X, A or B passes 2.82 and the scaled ones stay below 46200 of fp16's
// 65504, while the second part reaches down to 2^-38 of the largest.  A product is
// hi hi + hi lo + lo hi on the matrix unit with fp32 sums (lo lo is 2^-22 of it).
//
// Layout: a row's 32 columns are 128 bytes, 64 of the first parts and 64 of the
// second, so a 128-byte stage of the loop holds both parts of 32 k and gives three
// products: 2/3 of the fetches, LDS writes and LDS reads of three products one
// after the other.  Every operand is read along its rows: X is kept with its
// transpose, and A and B are symmetric (tiles on and above the diagonal are computed,
// and written twice).  Sides are padded with zeros to 32.
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
// sum of the squares of one matrix, in 64 bits: parts[z][block]
template <int DT>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const void* G, int64_t mn, double* parts) {
    typedef typename elem_of<DT>::type E;
    constexpr int V = kVec<DT>;
    __shared__ double red[4];
    const E* g = (const E*)G + (int64_t)blockIdx.y * mn;
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

// 64 x 64 of G / |G| in two parts, as they lie in G (to `as`) and transposed (to
// `across`); all NaN if G holds a NaN or an infinity.  mp, np: the padded sides.
template <int DT>
__global__ __launch_bounds__(256) void ortho_split_kernel(const void* G, int m, int n, int mp, int np,
                                                          const double* parts, int nparts, uint16_t* as, uint16_t* across) {
    typedef typename elem_of<DT>::type E;
    __shared__ double red[4];
    __shared__ float tile[64][65];
    const int64_t z = blockIdx.y;
    const int t = threadIdx.x;
    double s = 0.0;
    for (int i = t; i < nparts; i += 256) s += parts[z * kNormBlocks + i];
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, 64);
    if ((t & 63) == 0) red[t >> 6] = s;
    __syncthreads();
    s = (red[0] + red[1]) + (red[2] + red[3]);
    const double factor = s == 0.0 ? 0.0 : s < __builtin_inf() ? (double)kScale / sqrt(s) : __builtin_nan("");
    const int tn = (np + 63) / 64, r0 = (int)(blockIdx.x / tn) * 64, c0 = (int)(blockIdx.x % tn) * 64;
    const E* g = (const E*)G + z * (int64_t)m * n;
    as += z * 2 * mp * np;
    across += z * 2 * mp * np;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int r = r0 + 4 * i + (t >> 6), c = c0 + (t & 63);
        tile[4 * i + (t >> 6)][t & 63] = r < m && c < n ? (float)((double)elem_f32<DT>(g[(int64_t)r * n + c]) * factor) : 0.0f;
    }
    __syncthreads();
    // 16 lanes a row of 4 values each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = 16 * i + (t >> 4), b = 4 * (t & 15);
        float v[4];
        u32x2_t hi, lo;
        if (r0 + a < mp && c0 + b < np) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = tile[a][b + e];
            split4(v, hi, lo);
            uint16_t* d = as + part_at(r0 + a, c0 + b, np);
            *(u32x2_t*)d = hi;
            *(u32x2_t*)(d + 32) = lo;
        }
        if (c0 + a < np && r0 + b < mp) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = tile[b + e][a];
            split4(v, hi, lo);
            uint16_t* d = across + part_at(c0 + a, r0 + b, mp);
            *(u32x2_t*)d = hi;
            *(u32x2_t*)(d + 32) = lo;
        }
    }
}

// ------------------------------------------------------------------ products
// acc = sum over nk stages of hi hi + hi lo + lo hi.  NB stages in LDS, all but
// the current one on their way.  A stage's three phases: hi hi (while the columns'
// second parts are read), hi lo (the rows'), the barrier that retires the stage's
// buffer and publishes the next, lo hi (the next stage's first parts, and the DMA of
// stage kt + NB into the retired buffer).  P: which of fb holds the first parts.
template <int BT, int NB>
struct Loop {
    static constexpr int TM = BT / 32, NM = TM * TM, OPB = BT * 128, STAGE = 2 * OPB, LA = RowSrc<BT>::PER_WAVE;
    f32x4_t (&acc)[TM][TM];
    char* smem;
    const RowSrc<BT>&sa, &sb;
    int nk, lane, wave, rowa, rowb;
    u32x4_t fa[2][TM], fb[2][TM];

    __device__ __forceinline__ char* at(int kt) const { return smem + (kt % NB) * STAGE; }
    template <int p>
    __device__ __forceinline__ u32x4_t read(const char* st, int row, int i) const {
        return read_frag16<BT, true>(st, row + 16 * i, p, lane);
    }
    __device__ __forceinline__ void issue(int kt) const {
        const i32x4_t ra = sa.rsrc(kt, nk), rb = sb.rsrc(kt, nk);
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
            spread<NM, TM, decltype(xc)::value>([&](auto i) { fb[P ^ 1][i] = read<1>(st + OPB, rowb, i); });
        });
        phase<1, TM, TM, false>(acc, fa[0], fb[P ^ 1], [&](auto xc) {
            spread<NM, TM, decltype(xc)::value>([&](auto i) { fa[1][i] = read<1>(st, rowa, i); });
        });
        wait_vm<(NB - 2) * 2 * LA>();  // this wave's DMA of stage kt + 1 has landed
        __syncthreads();               // ... every wave's; and every read of stage kt is done
        fence_sched();
        const i32x4_t ra = sa.rsrc(kt + NB, nk), rb = sb.rsrc(kt + NB, nk);
        const uint32_t l = lds_addr(st);
        phase<1, TM, TM, false>(acc, fa[1], fb[P], [&](auto xc) {
            constexpr int x = decltype(xc)::value;
            spread<NM, 2 * LA, x>([&](auto d) {
                if constexpr (decltype(d)::value < LA) sa.one(ra, l, kt + NB, wave, d);
                else sb.one(rb, l + OPB, kt + NB, wave, d - LA);
            });
            spread<NM, 2 * TM, x>([&](auto r) {
                constexpr int i = decltype(r)::value / 2;
                if constexpr (decltype(r)::value % 2 == 0) fb[P ^ 1][i] = read<0>(nx + OPB, rowb, i);
                else fa[0][i] = read<0>(nx, rowa, i);
            });
        });
    }
    __device__ __forceinline__ void run() {
        for (int kt = 0; kt < NB; ++kt) issue(kt);
        wait_vm<(NB - 1) * 2 * LA>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            fa[0][i] = read<0>(smem, rowa, i);
            fb[0][i] = read<0>(smem + OPB, rowb, i);
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

enum OrthoOp { kGram, kPoly, kUpdate };

struct OrthoK {
    const uint16_t* A;  // (rows, K): rows of the result
    const uint16_t* B;  // (cols, K): its columns
    const uint16_t* C;  // (rows, cols): what the polynomial adds (kPoly: A, kUpdate: X)
    uint16_t* D;        // (rows, cols), the result
    uint16_t* Dt;       // (cols, rows), the same transposed (D itself where it is symmetric)
    void* out;          // or, of the last step, T
    int rows, cols, K;  // padded
    int m, n;           // of out: (rows, cols) without padding, or (cols, rows) of a tall G
    int tall;
    int tiles;          // of one matrix
};

// DT: 3 = in two parts, else T of the last step's result
template <int OP, int DT, int BT, int NB>
__global__ __launch_bounds__(NT, NB * BT * 256 <= 80 * 1024 ? 2 : 1) void ortho_kernel(OrthoK a) {
    constexpr bool SYM = OP != kUpdate, LAST = DT < 3;
    typedef Loop<BT, NB> L;
    constexpr int TM = L::TM;
    __shared__ __attribute__((aligned(1024))) char smem[NB * L::STAGE];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int w = xcd_remap((int)blockIdx.x, (int)gridDim.x);
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
    RowSrc<BT> sa, sb;
    sa.init(a.A + (int64_t)z * 2 * a.rows * a.K, a.K * 4, a.K * 4, m0, a.rows, lane);
    sb.init(a.B + (int64_t)z * 2 * a.cols * a.K, a.K * 4, a.K * 4, n0, a.cols, lane);
    f32x4_t acc[TM][TM];
    L loop{acc, smem, sa, sb, a.K / 32, lane, wave, wm * (BT / 2), wn * (BT / 2)};
    loop.run();

    // 32 rows of the wave's columns at a time pass through LDS, so that C is read and
    // the results are written by whole rows of 16 bytes a lane (8 bytes a lane straight
    // from the accumulators' layout: 45 us a 256 x 256 tile on an idle chip).  All of it
    // is the wave's own: no barrier.  Rows are of W bytes; of the transposed result 32
    // rows are 128 bytes of each column.
    constexpr int H = BT / 2, W = BT * 2, CPR = W / 16, NCH = 32 * CPR / 64;
    const int64_t size = (int64_t)z * 2 * a.rows * a.cols;
    const uint16_t* C = a.C + size;
    uint16_t *D = a.D + size, *Dt = a.Dt + size;
    char *direct = smem + wave * (128 * BT), *across = direct + 32 * W;
    const int wr = m0 + wm * H, wc = n0 + wn * H;
    // 16-byte piece of 32 columns' 128 bytes, by row: neighbouring rows in other banks
    const auto slot = [](int row, int piece) { return (piece ^ (row & 7)) << 4; };
    __syncthreads();  // every wave is done with the last stage
    u32x4_t cr[NCH];
    const auto load_c = [&](int r0) {
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
            const int row = (q * 64 + lane) / CPR, ch = (q * 64 + lane) % CPR;
            cr[q] = r0 + row < a.rows && wc + ch / 8 * 32 < a.cols
                        ? *(const u32x4_t*)(C + part_at(r0 + row, wc, a.cols) + ch * 8) : u32x4_t{0, 0, 0, 0};
        }
    };
    if constexpr (OP != kGram) load_c(wr);
#pragma unroll
    for (int h = 0; h < TM / 2; ++h) {
        const int r0 = wr + 32 * h;
        if (r0 >= a.rows) break;
        if constexpr (OP != kGram) {
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
                float v[4];
                if constexpr (OP == kGram) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * kUnscale;
                } else {
                    float x[4];
                    join4(*ph, *pl, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = OP == kPoly ? kB * x[e] + kC * (acc[i][j][e] * kUnscale) : kA * x[e] + acc[i][j][e] * kUnscale;
                }
                if constexpr (LAST) {
                    typedef typename elem_of<LAST ? DT : 2>::type E;
                    E* out = (E*)a.out + (int64_t)z * a.m * a.n;
                    const int r = r0 + row, c = wc + 16 * j + 4 * g;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int orow = a.tall ? c + e : r, col = a.tall ? r : c + e;
                        if (orow < a.m && col < a.n) out[(int64_t)orow * a.n + col] = f32_elem<LAST ? DT : 2>(v[e] * kUnscale);
                    }
                } else {
                    u32x2_t hi, lo;
                    split4(v, hi, lo);
                    *ph = hi;
                    *pl = lo;
                    if (!SYM || tm != tn) {
                        const int c = 16 * j + 4 * g + (lane & 3), pr = 2 * ii + ((lane & 15) >> 3);
                        char* to = across + c * 128 + ((lane >> 2) & 1) * 8;
                        *(u32x2_t*)(to + slot(c, pr)) = transpose4(hi, lane);
                        *(u32x2_t*)(to + slot(c, pr + 4)) = transpose4(lo, lane);
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (!LAST) {
#pragma unroll
            for (int q = 0; q < NCH; ++q) {
                const int row = (q * 64 + lane) / CPR, ch = (q * 64 + lane) % CPR;
                const u32x4_t d = *(const u32x4_t*)(direct + row * W + (ch >> 3) * 128 + slot(row, ch & 7));
                if (r0 + row < a.rows && wc + ch / 8 * 32 < a.cols)
                    *(u32x4_t*)(D + part_at(r0 + row, wc, a.cols) + ch * 8) = d;
            }
            if (!SYM || tm != tn) {
#pragma unroll
                for (int q = 0; q < H / 8; ++q) {
                    const int c = 8 * q + (lane >> 3), ch = lane & 7;
                    const u32x4_t d = *(const u32x4_t*)(across + c * 128 + slot(c, ch));
                    if (wc + c < a.cols) *(u32x4_t*)(Dt + part_at(wc + c, r0, a.rows) + ch * 8) = d;
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t padded(int64_t n) { return (n + 31) / 32 * 32; }

// 4096 x 4096 (128 stages, bf16): A 328 / 219 / 175 / 231 us with tiles of 64 / 128 /
// 192 / 256, the update 449 / 330 / 366 / 281; 512 x 1024: A 11.4 / 25 / 42 / 66, the
// update 8.3 / 18 / 35 / 50; 16 of 1000 x 1024: A 89 / 79 / 101 / 91, update 183 / 132 / 176 / 115.
constexpr TileTimes kTiles[] = {{64, 512, 3.4, 0.25, 0.3, 0.63}, {128, 512, 11, 0.43, 0.6, 1.29},
                                {192, 256, 26, 0.5, 1.17, 1.17}, {256, 256, 34, 1.0, 1.93, 1.93}};

int64_t tiles_of(const OrthoK& k, bool sym, int bt) {
    const int64_t tm = (k.rows + bt - 1) / bt, tn = (k.cols + bt - 1) / bt;
    return sym ? tm * (tm + 1) / 2 : tm * tn;
}

template <int OP, int DT>
void product(OrthoK k, int64_t Z, hipStream_t s) {
    const int bt = pick_tile(kTiles, k.K / 32, [&](int bt) { return Z * tiles_of(k, OP != kUpdate, bt); });
    log_choice("orthogonalize: %d x %d x %d, tiles of %d", k.rows, k.cols, k.K, bt);
    k.tiles = (int)tiles_of(k, OP != kUpdate, bt);
    const unsigned grid = (unsigned)(k.tiles * Z);
    if (bt == 64) ortho_kernel<OP, DT, 64, 4><<<grid, NT, 0, s>>>(k);
    else if (bt == 128) ortho_kernel<OP, DT, 128, 2><<<grid, NT, 0, s>>>(k);
    else if (bt == 192) ortho_kernel<OP, DT, 192, 3><<<grid, NT, 0, s>>>(k);
    else ortho_kernel<OP, DT, 256, 2><<<grid, NT, 0, s>>>(k);
}

template <int DT>
hipError_t ortho_run(const OrthoArgs& o, void* ws, hipStream_t s) {
    const bool tall = o.m > o.n;
    const int64_t mp = padded(o.m), np = padded(o.n), Z = o.batch, mn = o.m * o.n, p = tall ? np : mp, q = tall ? mp : np;
    char* w = (char*)ws;
    double* parts = (double*)w;
    w += align256((size_t)Z * kNormBlocks * 8);
    uint16_t *X[2], *Xt[2];  // (p, q) and (q, p)
    for (uint16_t** x : {&X[0], &X[1], &Xt[0], &Xt[1]}) {
        *x = (uint16_t*)w;
        w += align256((size_t)Z * 4 * p * q);
    }
    uint16_t* A = (uint16_t*)w;
    uint16_t* B = (uint16_t*)(w + align256((size_t)Z * 4 * p * p));
    const int nparts = (int)std::min<int64_t>(kNormBlocks, (mn + 8191) / 8192);
    ortho_norm_kernel<DT><<<dim3(nparts, (unsigned)Z), 256, 0, s>>>(o.G, mn, parts);
    const int64_t tiles = ((mp + 63) / 64) * ((np + 63) / 64);
    ortho_split_kernel<DT><<<dim3((unsigned)tiles, (unsigned)Z), 256, 0, s>>>(
        o.G, (int)o.m, (int)o.n, (int)mp, (int)np, parts, nparts, tall ? Xt[0] : X[0], tall ? X[0] : Xt[0]);
    OrthoK k;
    k.m = (int)o.m;
    k.n = (int)o.n;
    k.tall = tall;
    k.out = o.out;
    for (int step = 0; step < o.steps; ++step) {
        const int x = step & 1, y = x ^ 1;
        k.rows = k.cols = (int)p;
        k.K = (int)q;
        k.A = k.B = X[x];
        k.C = A;
        k.D = k.Dt = A;
        product<kGram, 3>(k, Z, s);
        k.K = (int)p;
        k.A = k.B = k.C = A;
        k.D = k.Dt = B;
        product<kPoly, 3>(k, Z, s);
        k.cols = (int)q;
        k.A = B;
        k.B = Xt[x];
        k.C = X[x];
        k.D = X[y];
        k.Dt = Xt[y];
        if (step + 1 == o.steps) product<kUpdate, DT>(k, Z, s);
        else product<kUpdate, 3>(k, Z, s);
    }
    return hipGetLastError();
}

}  // namespace

size_t orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n) {
    const int64_t mp = padded(m), np = padded(n), p = mp < np ? mp : np;
    return align256((size_t)batch * kNormBlocks * 8) + 4 * align256((size_t)batch * 4 * mp * np) +
           2 * align256((size_t)batch * 4 * p * p);
}

hipError_t launch_orthogonalize(const OrthoArgs& a, int dt, void* ws, hipStream_t s) {
    return dt == 0 ? ortho_run<0>(a, ws, s) : dt == 1 ? ortho_run<1>(a, ws, s) : ortho_run<2>(a, ws, s);
}

}  // namespace omm
