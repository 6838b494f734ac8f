// 8-bit products with a scale for each token and channel.
//
//   quantise:  scale[m] = amax_k |x[m, k]| / 127,  q[m, k] = 127 x[m, k] / amax, to the nearest integer (ties to even)
//   product:   Y[m, n] = T( sum_k a[m, k] b[n, k] * a_scale[m] * b_scale[n] + bias[n] )
//
// The sum is exact in int32 (K <= 131071 values of at most 128 * 128).  Both
// operands have k contiguous, so a tile of 128 bytes of k is the bf16 kernels'
// tile byte for byte.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm16_core.hpp"
#include "kernels.hpp"
#include "stream_core.hpp"

namespace omm {

namespace {

using namespace core16;

// ------------------------------------------------------------------ quantisation
// A row's values pass through registers once: their largest magnitude (as bits: a
// NaN is larger than every number), then the quotients.
struct QuantArgs {
    const void* X;  // (M, K)
    int8_t* Q;      // (M, ldq), columns past K zeroed
    float* scale;   // (M)
    int64_t M, ldq;
    int K;
};

typedef u32x2_t u32x2_u1 __attribute__((aligned(1)));
typedef uint32_t u32_u1 __attribute__((aligned(1)));

// 127 x / amax to the nearest integer.  x * inv is within 1.6e-5 of it (two
// roundings of values up to 127), so only what lies closer than that to the
// border of two steps is divided in 64 bits.
__device__ __forceinline__ float quantise(float x, float amax, float inv, bool tiny) {
    const float t = x * inv, q = rintf(t);
    if (tiny || fabsf(t - q) > 0.49996f) return (float)rint((double)x * 127.0 / (double)amax);
    return q;
}
template <int V>
__device__ __forceinline__ void quantise_store(int8_t* q, const float* f, int n, float amax, float inv, bool tiny) {
    uint32_t w[V / 4] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) w[i / 4] |= ((uint32_t)(int)quantise(f[i], amax, inv, tiny) & 255u) << (8 * (i & 3));
    if (n >= V) {
        if constexpr (V == 8)
            *(u32x2_u1*)q = u32x2_t{w[0], w[1]};
        else
            *(u32_u1*)q = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) q[i] = (int8_t)(w[i / 4] >> (8 * (i & 3)));
    }
}

// NW waves a row, C 16-byte chunks a lane (C = 0: rows of any length, read twice)
template <int DT, int NW, int C>
__global__ __launch_bounds__(NW <= 4 ? 256 : 64 * NW) void quantise_kernel(QuantArgs a) {
    typedef typename elem_of<DT>::type E;
    constexpr int V = kVec<DT>, NL = 64 * NW, ROWS = NW <= 4 ? 4 / NW : 1;
    __shared__ uint32_t part[NW > 1 ? NW : 1];
    const int t = threadIdx.x, l = t % NL, K = a.K;
    const int64_t m = (int64_t)blockIdx.x * ROWS + t / NL;
    const bool here = m < a.M;
    const E* row = (const E*)a.X + (here ? m : a.M - 1) * K;
    u32x4_t v[C ? C : 1];
    uint32_t mx = 0;
    const auto largest = [&](u32x4_t w) {
        float f[V];
        unpack16<DT>(w, f);
#pragma unroll
        for (int i = 0; i < V; ++i) mx = max(mx, __float_as_uint(f[i]) & 0x7fffffffu);
    };
    if constexpr (C) {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = load16_first(row + min((c * NL + l) * V, K), max(0, K - (c * NL + l) * V));
#pragma unroll
        for (int c = 0; c < C; ++c) largest(v[c]);
    } else {
        for (int64_t e = (int64_t)l * V; e < K; e += NL * V) largest(load16_first(row + e, (int)min((int64_t)V, K - e)));
    }
    mx = wave_max_u32(mx);
    if constexpr (NW > 1) {
        if ((t & 63) == 0) part[t >> 6] = mx;
        __syncthreads();
        mx = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) mx = max(mx, part[w]);
    }
    if (!here) return;
    // a row that holds a NaN or an infinity: its scale is NaN and its values 0
    const bool finite = mx < 0x7f800000u;
    const float amax = __uint_as_float(mx), s = finite ? amax / 127.0f : __builtin_nanf("");
    const bool tiny = finite && mx && amax < 0x1p-100f;
    const float inv = finite && mx && !tiny ? 127.0f / amax : 0.0f;
    if (l == 0) a.scale[m] = s;
    int8_t* q = a.Q + m * a.ldq;
    const auto out = [&](int64_t e, u32x4_t w) {
        float f[V];
        unpack16<DT>(w, f);
        if (!finite || !mx) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = 0.0f;
        }
        quantise_store<V>(q + e, f, (int)min((int64_t)V, a.ldq - e), amax, inv, tiny);
    };
    if constexpr (C) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * NL + l) * V;
            if (e < a.ldq) out(e, v[c]);
        }
    } else {
        for (int64_t e = (int64_t)l * V; e < a.ldq; e += NL * V) {
            const int n = (int)max((int64_t)0, min((int64_t)V, K - e));
            out(e, load16_first(row + min(e, (int64_t)K), n));
        }
    }
}

template <int DT>
hipError_t quantise_run(const QuantArgs& a, hipStream_t s) {
    constexpr int V = kVec<DT>;
    const auto go = [&](auto kernel, int nw) {
        const int rows = nw <= 4 ? 4 / nw : 1;
        constexpr int64_t kMost = 1 << 21;  // rows a launch: a grid has at most 2^32 - 1 threads
        for (int64_t m = 0; m < a.M; m += kMost) {
            QuantArgs p = a;
            p.X = (const typename elem_of<DT>::type*)a.X + m * a.K;
            p.Q = a.Q + m * a.ldq;
            p.scale = a.scale + m;
            p.M = a.M - m < kMost ? a.M - m : kMost;
            kernel<<<dim3((unsigned)((p.M + rows - 1) / rows)), nw <= 4 ? 256 : 64 * nw, 0, s>>>(p);
        }
    };
    const int64_t chunks = (a.ldq + V - 1) / V;  // of 16 bytes of X
    if (chunks <= 64) go(quantise_kernel<DT, 1, 1>, 1);
    else if (chunks <= 128) go(quantise_kernel<DT, 1, 2>, 1);
    else if (chunks <= 256) go(quantise_kernel<DT, 4, 1>, 4);
    else if (chunks <= 512) go(quantise_kernel<DT, 4, 2>, 4);
    else if (chunks <= 1024) go(quantise_kernel<DT, 4, 4>, 4);
    else if (chunks <= 4096) go(quantise_kernel<DT, 16, 4>, 16);
    else go(quantise_kernel<DT, 16, 0>, 16);
    return hipGetLastError();
}

hipError_t quantise_dt(const QuantArgs& a, int dt, hipStream_t s) {
    return dt == 0 ? quantise_run<0>(a, s) : dt == 1 ? quantise_run<1>(a, s) : quantise_run<2>(a, s);
}

// ------------------------------------------------------------------ product
struct ProductArgs {
    const int8_t* a;       // (M, lda)
    const int8_t* b;       // (N, K)
    const float* a_scale;  // (M)
    const float* b_scale;  // (N)
    const void* bias;      // (N) of T or nullptr
    void* Y;               // (M, N) of T
    int64_t M, N, lda;
    int K;
};

// Four neighbouring results of a row
template <int DT>
__device__ __forceinline__ void scaled4(const i32x4_t& acc, float sa, const float (&sb)[4], const float (&bias)[4],
                                        float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)acc[e] * sa * sb[e] + bias[e];
}
template <int DT>
__device__ __forceinline__ void store4(void* Y, int64_t at, const float (&v)[4], int n) {
    typedef typename elem_of<DT>::type E;
    E* y = (E*)Y + at;
    if (n >= 4) {
        if constexpr (DT == 2) {
            typedef f32x4_t f32x4_u4 __attribute__((aligned(4)));
            *(f32x4_u4*)y = f32x4_t{v[0], v[1], v[2], v[3]};
        } else {
            typedef u32x2_t u32x2_u2 __attribute__((aligned(2)));
            *(u32x2_u2*)y = u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) y[e] = f32_elem<DT>(v[e]);
    }
}

// BT x BT tiles, 4 waves of (BT / 2)^2.  MODE 0: whole tiles by DMA; 1: ragged
// ones by DMA (16-byte aligned rows); 2: rows at any byte, through registers.
template <int BT, int DT, int MODE>
__global__ __launch_bounds__(NT, BT == 128 ? 2 : 1) void int8_tile_kernel(ProductArgs a, int tiles_m, int tiles_n) {
    constexpr int TM = BT / 32, TN = BT / 32, OP = BT * 128, STAGE = 2 * OP;
    __shared__ __attribute__((aligned(1024))) char smem0[STAGE];
    __shared__ __attribute__((aligned(1024))) char smem1[STAGE];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    grouped_order(xcd_remap((int)blockIdx.x, (int)gridDim.x), tiles_m, tiles_n, 4, tm, tn);
    const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
    const int nk = (a.K + 127) / 128;
    f32x4_t acc[TM][TN];
    if constexpr (MODE < 2) {
        DmaSrc<BT, true, 1> sa, sb;
        sa.init(a.a, a.lda, m0, a.M, a.K, lane);
        sb.init(a.b, a.K, n0, a.N, a.K, lane);
        mainloop_dma16<BT, BT, 3, true, true, MODE == 1>(acc, smem0, smem1, sa, sb, nk, lane, wm, wn, wave);
    } else {
        i32x4_t sum[TM][TN] = {};
        constexpr int NC = BT * 8 / NT;  // 16-byte chunks of an operand a thread
        u32x4_t r[2][NC];
        const auto load = [&](int kt) {
#pragma unroll
            for (int i = 0; i < 2 * NC; ++i) {
                const int row = (t >> 3) + 32 * (i % NC);
                const int k = kt * 128 + 16 * (t & 7), n = min(16, a.K - k);
                const bool isb = i >= NC;
                const int64_t at = (isb ? n0 : m0) + row;
                u32x4_t v = {0, 0, 0, 0};
                if (at < (isb ? a.N : a.M) && n > 0) {
                    const int8_t* p = (isb ? a.b + at * a.K : a.a + at * a.lda) + k;
                    if (n == 16) {
                        typedef u32x4_t u32x4_u1 __attribute__((aligned(1)));
                        v = *(const u32x4_u1*)p;
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e < n) v[e >> 2] |= (uint32_t)(uint8_t)p[e] << (8 * (e & 3));
                    }
                }
                r[i / NC][i % NC] = v;
            }
        };
        load(0);
        for (int kt = 0; kt < nk; ++kt) {
            char* s = kt & 1 ? smem1 : smem0;
#pragma unroll
            for (int i = 0; i < 2 * NC; ++i)
                *(u32x4_t*)(s + (i / NC) * OP + kmaj_off<BT>((t >> 3) + 32 * (i % NC), t & 7)) = r[i / NC][i % NC];
            __syncthreads();  // (the other buffer's readers passed the barrier before)
            if (kt + 1 < nk) load(kt + 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4_t fa[TM], fb[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i) fa[i] = read_frag16<BT, true>(s, wm * (BT / 2) + 16 * i, h, lane);
#pragma unroll
                for (int j = 0; j < TN; ++j) fb[j] = read_frag16<BT, true>(s + OP, wn * (BT / 2) + 16 * j, h, lane);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        sum[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, fb[j]),
                                                                          __builtin_bit_cast(i32x4_t, fa[i]), sum[i][j], 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_bit_cast(f32x4_t, sum[i][j]);
    }
    typedef typename elem_of<DT>::type E;
    float sa[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = a.a_scale[min(m0 + wm * (BT / 2) + 16 * i + (lane & 15), a.M - 1)];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t n = n0 + wn * (BT / 2) + 16 * j + 4 * (lane >> 4);
        if (n >= a.N) continue;
        float sb[4], bias[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sb[e] = a.b_scale[min(n + e, a.N - 1)];
            bias[e] = a.bias ? elem_f32<DT>(((const E*)a.bias)[min(n + e, a.N - 1)]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = m0 + wm * (BT / 2) + 16 * i + (lane & 15);
            float v[4];
            scaled4<DT>(__builtin_bit_cast(i32x4_t, acc[i][j]), sa[i], sb, bias, v);
            if (m < a.M) store4<DT>(a.Y, m * a.N + n, v, (int)min((int64_t)4, a.N - n));
        }
    }
}

// no contraction: Y = bias
template <int DT>
__global__ __launch_bounds__(256) void int8_bias_kernel(ProductArgs a) {
    typedef typename elem_of<DT>::type E;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < a.M * a.N; n += (int64_t)gridDim.x * 256) {
        const int64_t c = n % a.N;
        // 0 a_scale b_scale: NaN where a scale is, as in a row that was not finite
        const float z = 0.0f * a.a_scale[n / a.N] * a.b_scale[c];
        ((E*)a.Y)[n] = f32_elem<DT>(z + (a.bias ? elem_f32<DT>(((const E*)a.bias)[c]) : 0.0f));
    }
}

template <int DT>
hipError_t product_run(const ProductArgs& a, hipStream_t s) {
    if (a.K == 0) {
        int8_bias_kernel<DT><<<dim3((unsigned)std::min<int64_t>((a.M * a.N + 255) / 256, 1 << 16)), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    const bool aligned = a.K % 16 == 0 && a.lda % 16 == 0 && (((uintptr_t)a.a | (uintptr_t)a.b) & 15) == 0;
    const auto tiles = [&](auto kernel, int bt) {
        const int64_t tm = (a.M + bt - 1) / bt, tn = (a.N + bt - 1) / bt;
        kernel<<<dim3((unsigned)(tm * tn)), NT, 0, s>>>(a, (int)tm, (int)tn);
    };
    if (!aligned) tiles(int8_tile_kernel<128, DT, 2>, 128);
    else if (a.M % 256 == 0 && a.N % 256 == 0 && a.K % 128 == 0 && (a.M / 256) * (a.N / 256) >= 256)
        tiles(int8_tile_kernel<256, DT, 0>, 256);
    else if (a.M % 128 == 0 && a.N % 128 == 0 && a.K % 128 == 0) tiles(int8_tile_kernel<128, DT, 0>, 128);
    else tiles(int8_tile_kernel<128, DT, 1>, 128);
    return hipGetLastError();
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t padded(int64_t K) { return (K + 15) / 16 * 16; }

}  // namespace

hipError_t launch_quantize_rows(const void* X, int8_t* Q, float* scale, int64_t M, int64_t K, int dt, hipStream_t s) {
    return quantise_dt({X, Q, scale, M, K, (int)K}, dt, s);
}

size_t int8_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N, bool quantise) {
    if (!quantise) return 0;
    return align256((size_t)M * 4) + align256((size_t)M * (size_t)padded(K));
}

hipError_t launch_int8_matmul(const Int8Args& x, int dt, void* ws, hipStream_t s) {
    ProductArgs a = {(const int8_t*)x.a, (const int8_t*)x.b, x.a_scale, x.b_scale, x.bias, x.Y, x.M, x.N, x.K, (int)x.K};
    if (x.a_kind >= 0) {
        float* scale = (float*)ws;
        int8_t* q = (int8_t*)ws + align256((size_t)x.M * 4);
        const int64_t ld = padded(x.K);
        const hipError_t e = quantise_dt({x.a, q, scale, x.M, ld, (int)x.K}, x.a_kind, s);
        if (e != hipSuccess) return e;
        a.a = q;
        a.lda = ld;
        a.a_scale = scale;
    }
    return dt == 0 ? product_run<0>(a, s) : dt == 1 ? product_run<1>(a, s) : product_run<2>(a, s);
}

}  // namespace omm
