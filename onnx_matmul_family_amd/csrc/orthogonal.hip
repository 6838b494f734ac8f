// Orthogonalised update: Newton-Schulz steps on a matrix (or a batch of them).
//
//   X = G / |G| (Frobenius);  `steps` times:  A = X X^T,  X <- a X + (b A + c A^2) X
//   (tall matrices: A = X^T X,  X <- a X + X (b A + c A^2): the same odd polynomial
//   of the singular values, over the shorter side)
//
// The steps multiply what is small in X by up to 3.44 each, roundings included, so
// X, A and B = b A + c A^2 are held to 22 bits: as two fp16 parts (value, and what
// its rounding leaves), scaled by 2^14.  Singular values stay below 1.21, so no
// entry of X, A or B passes 2.82 and the scaled ones stay below 46200 of fp16's
// 65504, while the second part reaches down to 2^-38 of the largest.  A product is
// hi hi + hi lo + lo hi on the matrix unit with fp32 sums (lo lo is 2^-22 of it).
// A and B are symmetric: tiles on and above the diagonal are computed and written twice.
//
// Everything but G and the result is padded with zeros to whole tiles in the workspace.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm16_core.hpp"
#include "kernels.hpp"
#include "stream_core.hpp"

namespace omm {

namespace {

using namespace core16;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 16384.0f, kUnscale = 1.0f / 16384.0f;
constexpr int kNormBlocks = 64;
constexpr int BT = 128;

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

// X = G / |G| in two parts, padded; all NaN if G holds a NaN or an infinity
template <int DT>
__global__ __launch_bounds__(256) void ortho_split_kernel(const void* G, int m, int n, int mp, int np,
                                                          const double* parts, int nparts, uint16_t* X) {
    typedef typename elem_of<DT>::type E;
    constexpr int V = kVec<DT>;
    __shared__ double factor_s;
    const int64_t z = blockIdx.y;
    if (threadIdx.x < 64) {
        double s = (int)threadIdx.x < nparts ? parts[z * kNormBlocks + threadIdx.x] : 0.0;
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, 64);
        if (threadIdx.x == 0) factor_s = s == 0.0 ? 0.0 : s < __builtin_inf() ? (double)kScale / sqrt(s) : __builtin_nan("");
    }
    __syncthreads();
    const double factor = factor_s;
    const E* g = (const E*)G + z * (int64_t)m * n;
    const int64_t plane = (int64_t)mp * np, per_row = np / V;
    uint16_t* hi = X + z * 2 * plane;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < mp * per_row; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / per_row), col = (int)(i % per_row) * V;
        const int k = row < m ? max(0, min(V, n - col)) : 0;
        float f[V];
        unpack16<DT>(load16_first(g + (k ? (int64_t)row * n + col : 0), k), f);
#pragma unroll
        for (int h = 0; h < V; h += 4) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = h + e < k ? (float)((double)f[h + e] * factor) : 0.0f;
            u32x2_t a, b;
            split4(v, a, b);
            *(u32x2_t*)(hi + (int64_t)row * np + col + h) = a;
            *(u32x2_t*)(hi + plane + (int64_t)row * np + col + h) = b;
        }
    }
}

// ------------------------------------------------------------------ products
// One operand of hi hi + hi lo + lo hi: a stage of k is three of the loop's, its
// part by LO (bit s: the s-th takes the second part).
template <class S, int LO>
struct PartSrc {
    static constexpr int PER_WAVE = S::PER_WAVE;
    S s;
    int64_t lo;  // bytes from the first part to the second
    __device__ __forceinline__ DmaCtx ctx(char* lds, int kt, bool live = true) const {
        const int k = kt / 3, part = kt - 3 * k;
        return DmaCtx{make_rsrc(s.base + (live ? (int64_t)k * s.step + ((LO >> part) & 1 ? lo : 0) : 0), live), lds_addr(lds)};
    }
    template <bool CHECKED>
    __device__ __forceinline__ void one(const DmaCtx& c, int kt, int wave, int j) const {
        s.template one<false>(c, 0, wave, j);
    }
};

enum OrthoOp { kGramWide, kGramTall, kPoly, kUpdateWide, kUpdateTall };

struct OrthoK {
    const uint16_t* A;  // rows of the result; [z][part][..]
    const uint16_t* B;  // its columns
    const uint16_t* C;  // what the polynomial adds (kPoly: A, kUpdate: X), laid out as the result
    uint16_t* D;        // the result in two parts
    void* out;          // or, of the last step, (m, n) of T
    int rows, cols, K;  // padded
    int m, n;
    int tiles;          // of one matrix
};

template <int OP, int DT>
__global__ __launch_bounds__(NT, 2) void ortho_kernel(OrthoK a) {
    constexpr bool SYM = OP <= kPoly, AK = OP != kGramTall, BK = OP != kGramTall && OP != kUpdateWide;
    constexpr bool LAST = DT < 3;
    constexpr int TM = BT / 32, TN = BT / 32, OPB = BT * KSTEP * 2, STAGE = 2 * OPB;
    __shared__ __attribute__((aligned(1024))) char smem0[STAGE];
    __shared__ __attribute__((aligned(1024))) char smem1[STAGE];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int w = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    const int z = w / a.tiles;
    int tm, tn, i = w - z * a.tiles;
    if constexpr (SYM) {
        // i-th of the tiles tn >= tm, row by row
        const int T = a.rows / BT;
        tm = 0;
        while (i >= T - tm) i -= T - tm++;
        tn = tm + i;
    } else {
        grouped_order(i, a.rows / BT, a.cols / BT, 4, tm, tn);
    }
    const int m0 = tm * BT, n0 = tn * BT;
    const int64_t aplane = (int64_t)a.rows * a.K, bplane = (int64_t)a.cols * a.K, cplane = (int64_t)a.rows * a.cols;
    PartSrc<DmaSrc<BT, AK>, 4> sa;
    PartSrc<DmaSrc<BT, BK>, 2> sb;
    sa.s.init(a.A + z * 2 * aplane, AK ? a.K : a.rows, m0, a.rows, a.K, lane);
    sb.s.init(a.B + z * 2 * bplane, BK ? a.K : a.cols, n0, a.cols, a.K, lane);
    sa.lo = aplane * 2;
    sb.lo = bplane * 2;
    f32x4_t acc[TM][TN];
    mainloop_dma16<BT, BT, 1, AK, BK, false>(acc, smem0, smem1, sa, sb, 3 * (a.K / KSTEP), lane, wm, wn, wave);

    const uint16_t* C = a.C + z * 2 * cplane;
    uint16_t* D = a.D + z * 2 * cplane;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = m0 + wm * (BT / 2) + 16 * i + (lane & 15);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int c = n0 + wn * (BT / 2) + 16 * j + 4 * (lane >> 4);
            const int64_t at = (int64_t)r * a.cols + c;
            float v[4];
            if constexpr (OP <= kGramTall) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * kUnscale;
            } else {
                float x[4];
                join4(*(const u32x2_t*)(C + at), *(const u32x2_t*)(C + cplane + at), x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = OP == kPoly ? kB * x[e] + kC * (acc[i][j][e] * kUnscale) : kA * x[e] + acc[i][j][e] * kUnscale;
            }
            if constexpr (LAST) {
                typedef typename elem_of<LAST ? DT : 2>::type E;
                E* out = (E*)a.out + (int64_t)z * a.m * a.n + (int64_t)r * a.n + c;
                if (r < a.m) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < a.n) out[e] = f32_elem<LAST ? DT : 2>(v[e] * kUnscale);
                }
            } else {
                u32x2_t hi, lo;
                split4(v, hi, lo);
                *(u32x2_t*)(D + at) = hi;
                *(u32x2_t*)(D + cplane + at) = lo;
                if (SYM && tm != tn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int64_t mirror = (int64_t)(c + e) * a.cols + r;
                        D[mirror] = (uint16_t)(hi[e >> 1] >> (16 * (e & 1)));
                        D[cplane + mirror] = (uint16_t)(lo[e >> 1] >> (16 * (e & 1)));
                    }
                }
            }
        }
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t tile_pad(int64_t n) { return (n + BT - 1) / BT * BT; }

template <int DT>
hipError_t ortho_run(const OrthoArgs& o, void* ws, hipStream_t s) {
    const int64_t mp = tile_pad(o.m), np = tile_pad(o.n), Z = o.batch, mn = o.m * o.n;
    const bool tall = o.m > o.n;
    const int64_t sp = tall ? np : mp;
    char* w = (char*)ws;
    double* parts = (double*)w;
    w += align256((size_t)Z * kNormBlocks * 8);
    uint16_t* X[2];
    for (auto& x : X) {
        x = (uint16_t*)w;
        w += align256((size_t)Z * 4 * mp * np);
    }
    uint16_t* A = (uint16_t*)w;
    uint16_t* B = (uint16_t*)(w + align256((size_t)Z * 4 * sp * sp));
    const int nparts = (int)std::min<int64_t>(kNormBlocks, (mn + 8191) / 8192);
    ortho_norm_kernel<DT><<<dim3(nparts, (unsigned)Z), 256, 0, s>>>(o.G, mn, parts);
    const int64_t chunks = mp * (np / kVec<DT>);
    ortho_split_kernel<DT><<<dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, 4096), (unsigned)Z), 256, 0, s>>>(
        o.G, (int)o.m, (int)o.n, (int)mp, (int)np, parts, nparts, X[0]);
    const int T = (int)(sp / BT), sym = T * (T + 1) / 2, all = (int)((mp / BT) * (np / BT));
    OrthoK k;
    k.m = (int)o.m;
    k.n = (int)o.n;
    k.out = o.out;
    for (int step = 0; step < o.steps; ++step) {
        const uint16_t* x = X[step & 1];
        uint16_t* y = X[(step + 1) & 1];
        k.rows = k.cols = (int)sp;
        k.tiles = sym;
        k.K = (int)(tall ? mp : np);
        k.A = k.B = x;
        k.C = nullptr;
        k.D = A;
        if (tall) ortho_kernel<kGramTall, 3><<<(unsigned)(sym * Z), NT, 0, s>>>(k);
        else ortho_kernel<kGramWide, 3><<<(unsigned)(sym * Z), NT, 0, s>>>(k);
        k.K = (int)sp;
        k.A = k.B = k.C = A;
        k.D = B;
        ortho_kernel<kPoly, 3><<<(unsigned)(sym * Z), NT, 0, s>>>(k);
        k.rows = (int)mp;
        k.cols = (int)np;
        k.tiles = all;
        k.A = tall ? x : B;
        k.B = tall ? B : x;
        k.C = x;
        k.D = y;
        const unsigned grid = (unsigned)(all * Z);
        const bool last = step + 1 == o.steps;
        if (tall && last) ortho_kernel<kUpdateTall, DT><<<grid, NT, 0, s>>>(k);
        else if (tall) ortho_kernel<kUpdateTall, 3><<<grid, NT, 0, s>>>(k);
        else if (last) ortho_kernel<kUpdateWide, DT><<<grid, NT, 0, s>>>(k);
        else ortho_kernel<kUpdateWide, 3><<<grid, NT, 0, s>>>(k);
    }
    return hipGetLastError();
}

}  // namespace

size_t orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n) {
    const int64_t mp = tile_pad(m), np = tile_pad(n), sp = m > n ? np : mp;
    return align256((size_t)batch * kNormBlocks * 8) + 2 * align256((size_t)batch * 4 * mp * np) +
           2 * align256((size_t)batch * 4 * sp * sp);
}

hipError_t launch_orthogonalize(const OrthoArgs& a, int dt, void* ws, hipStream_t s) {
    return dt == 0 ? ortho_run<0>(a, ws, s) : dt == 1 ? ortho_run<1>(a, ws, s) : ortho_run<2>(a, ws, s);
}

}  // namespace omm
