// 8-bit products with a scale for each token and channel.
//
//   quantise:  scale[m] = amax_k |x[m, k]| / 127,  q[m, k] = 127 x[m, k] / amax, to the nearest integer (ties to even)
//   product:   Y[m, n] = T( sum_k a[m, k] b[n, k] * a_scale[m] * b_scale[n] + bias[n] )
//
// The sum is exact in int32 (K <= 131071 values of at most 128 * 128).  Both
// operands have k contiguous, so a tile of 128 bytes of k is the bf16 kernels'
// tile byte for byte.
//
// What bounds it: few rows, the one read of b (1 row, 4096 x 4096: 16.8 MB in 6.5 us,
// 2.6 TB/s, as a launch and a first load take half of that; 1 row, 8192 x 8192: 4.0 TB/s).
// Tiles that are few, what one CU fetches (73 GB/s measured, whatever the loop: 4096 x 8192 x 128
// in 128 tiles of 64, 1 MB each, 14.3 us, half the CUs idle: K is not split over workgroups).
// Many tiles, the matrix unit: 8192 x 4096 x 8192 in 237 us beside other work and 229 alone,
// 2.3 to 2.4 POP/s, where the library's int8 product of 8192^3 reaches 2.5.  Quantising is one
// read and one write: 8192 x 4096 bf16 in 17.6 us, 5.7 TB/s of the 6.06 that a plain copy
// kernel reaches (torch's of 1 GiB: 5.13), 8192 x 4095 in 18.1.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.hpp"
#include "row_loop.hpp"
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

// Largest magnitude, as bits of fp32; of 16-bit types as their own bits, two at a time
template <int DT>
struct RowMax {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    uint32_t m = 0;
    __device__ __forceinline__ void add(u32x4_t v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == 2)
                m = max(m, v[i] & 0x7fffffffu);
            else
                m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, m),
                                                                           __builtin_bit_cast(u16x2_t, v[i] & 0x7fff7fffu)));
        }
    }
    __device__ __forceinline__ uint32_t bits() const {
        if constexpr (DT == 2) return m;
        else return __float_as_uint(from_bits<DT>((uint16_t)max(m & 0xffffu, m >> 16)));
    }
};

// 127 x / amax to the nearest integer, as bytes.  x * inv is within 7.6e-6 of it (127 /
// amax is rounded once, the product not at all), and adding 1.5 2^23 rounds that to an
// integer, whose two's complement is then the low bits.  What lies within 1e-5 of the
// border h / 2 (h odd) of two steps is decided by the sign of 254 x - h amax, exactly: with
// p = fp32(h amax), 254 x - p and h amax - p both fit fp32 (halves of 2^-8 of them
// here, so that neither passes its range; amax is 2^-100 or more).
template <int V>
__device__ __forceinline__ void quantise(const float* f, float amax, float inv, uint32_t (&w)[V / 4]) {
    constexpr float kRound = 12582912.0f;
    float r[V], off = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        r[i] = fmaf(f[i], inv, kRound);
        off = fmaxf(off, fabsf(fmaf(f[i], inv, kRound - r[i])));
    }
    if (off > 0.49999f) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float q = r[i] - kRound, d = fmaf(f[i], inv, -q);
            const float h = 2.0f * q + (d > 0.0f ? 1.0f : -1.0f), p = h * 0x1p-9f * amax;
            const float x = fmaf(f[i], 254.0f * 0x1p-9f, -p), y = fmaf(h * 0x1p-9f, amax, -p);
            const float below = 0.5f * h - 0.5f, even = 2.0f * rintf(0.25f * h);
            if (fabsf(d) > 0.49999f) r[i] = kRound + (x > y ? below + 1.0f : x < y ? below : even);
        }
    }
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const float* b = r + 4 * i;
        w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(__float_as_uint(b[3]), __float_as_uint(b[2]), 0x0400u),
                                     __builtin_amdgcn_perm(__float_as_uint(b[1]), __float_as_uint(b[0]), 0x0400u), 0x05040100u);
    }
}
// What a row's largest magnitude (as bits) makes of it.  A row that holds a NaN or
// an infinity: scale NaN and values 0.
struct RowScale {
    float amax, inv, scale;
    bool zero, tiny;
    __device__ __forceinline__ explicit RowScale(uint32_t mx) {
        const bool finite = mx < 0x7f800000u;
        amax = __uint_as_float(mx);
        scale = finite ? amax / 127.0f : __builtin_nanf("");
        zero = !finite || mx == 0;
        tiny = amax < 0x1p-100f;  // then 2^60 times all of it, which no fp32 is too small for
        if (tiny) amax *= 0x1p60f;
        inv = 127.0f / amax;
    }
    template <int V>
    __device__ __forceinline__ void bytes(float* f, uint32_t (&w)[V / 4]) const {
        if (tiny) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] *= 0x1p60f;
        }
        if (zero) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) w[i] = 0;
        } else {
            quantise<V>(f, amax, inv, w);
        }
    }
};

// NW waves a row, C 16-byte chunks a lane (C = 0: rows of any length, read twice).  The
// last chunk ends with the row (its first values are the one's before it too, and written twice).
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
    RowMax<DT> largest;
    const auto load = [&](int64_t e) { return K >= V ? load16(row + min(e, (int64_t)(K - V))) : load16_first(row, K); };
    if constexpr (C) {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = load((c * NL + l) * V);
#pragma unroll
        for (int c = 0; c < C; ++c) largest.add(v[c]);
    } else {
        for (int64_t e = (int64_t)l * V; e < K; e += NL * V) largest.add(load(e));
    }
    uint32_t mx = wave_max_u32(largest.bits());
    if constexpr (NW > 1) {
        if ((t & 63) == 0) part[t >> 6] = mx;
        __syncthreads();
        mx = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) mx = max(mx, part[w]);
    }
    if (!here) return;
    const RowScale rs(mx);
    if (l == 0) a.scale[m] = rs.scale;
    int8_t* q = a.Q + m * a.ldq;
    const auto out = [&](int64_t e, u32x4_t v) {
        float f[V];
        uint32_t w[V / 4];
        unpack16<DT>(v, f);
        rs.bytes<V>(f, w);
        if (K >= V) {
            int8_t* d = q + min(e, (int64_t)(K - V));
            if constexpr (V == 8) *(u32x2_u1*)d = u32x2_t{w[0], w[1]};
            else *(u32_u1*)d = w[0];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < K) q[i] = (int8_t)(w[i / 4] >> (8 * (i & 3)));
        }
    };
    if constexpr (C) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * NL + l) * V;
            if (e < K) out(e, v[c]);
        }
    } else {
        for (int64_t e = (int64_t)l * V; e < K; e += NL * V) out(e, load(e));
    }
    for (int64_t e = K + l; e < a.ldq; e += NL) q[e] = 0;
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
    const int64_t chunks = ((int64_t)a.K + V - 1) / V;  // of 16 bytes of X
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
    const int8_t* b;       // (N, ldb)
    const float* a_scale;  // (M)
    const float* b_scale;  // (N)
    const void* bias;      // (N) of T or nullptr
    void* Y;               // (M, N) of T
    int64_t M, N, lda, ldb;
    int K;
};

typedef u32x4_t u32x4_u1 __attribute__((aligned(1)));
// 16 bytes at p, zeros from the n-th on, as the whole words that hold them, shifted into
// place: no branch, as every load by itself would be a round trip.  p is inside the operand
// for any n.  (A word that holds a byte of the operand is of its memory.)
__device__ __forceinline__ u32x4_t bytes16(const int8_t* p, int n) {
    const uint32_t by = (uint32_t)((uintptr_t)p & 3);
    const int last = (int)by + max(min(n, 16), 1) - 1;  // byte of the last word, from the first word's start
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = *(const uint32_t*)(p - by + min(4 * j, last & ~3));
    u32x4_t v;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        v[d] = __builtin_amdgcn_alignbyte(w[d + 1], w[d], by);
        if (n < 4 * d + 4) v[d] &= n <= 4 * d ? 0u : (1u << (8 * (n - 4 * d))) - 1u;
    }
    return v;
}
__device__ __forceinline__ i32x4_t mfma_i8(u32x4_t a, u32x4_t b, i32x4_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// Scales and bias of four neighbouring columns (past the last: of the last)
template <int DT>
struct Columns {
    float scale[4], bias[4];
    __device__ __forceinline__ Columns(const ProductArgs& a, int64_t n) {
        typedef typename elem_of<DT>::type E;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            scale[e] = a.b_scale[min(n + e, a.N - 1)];
            bias[e] = a.bias ? elem_f32<DT>(((const E*)a.bias)[min(n + e, a.N - 1)]) : 0.0f;
        }
    }
    __device__ __forceinline__ void values(const i32x4_t& acc, float sa, float (&v)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[e] * sa * scale[e] + bias[e];
    }
};
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

// ------------------------------------------------------------------ few rows
// Up to 64 rows against 16 NF columns a workgroup at a time: one read of b, of which
// each of 8 waves takes every 8th 128 bytes of k (the sums of integers join in LDS in
// any order).  A wave loads 128 bytes of a row by 8 neighbouring lanes, 8 rows at a
// time (in the operands' order every lane would be a line of its own), and the
// operands take their places through LDS of the wave's own.  Any alignment, any K.
// AK: -1, a is int8; else rows of that type (few), which every workgroup quantises
// for itself while the first of b is on its way.
struct FewArgs {
    ProductArgs p;
    const void* X;  // AK >= 0: (M, K)
    int kpad;       // K to whole 128 bytes
};
constexpr int kFewWaves = 8;

template <int DT, int NF, int MG, int U, int AK>
__global__ __launch_bounds__(64 * kFewWaves) void int8_few_kernel(FewArgs f) {
    constexpr int XG = AK < 0 ? MG : 0;  // groups of 16 rows that are loaded as b is
    constexpr int UNIT = 128;            // 16-byte pieces of 16 rows
    extern __shared__ u32x4_t smem[];
    ProductArgs a = f.p;
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    if constexpr (AK < 0) {  // 16 MG rows of more
        const int64_t m0 = (int64_t)blockIdx.y * (16 * MG);
        a.a += m0 * a.lda;
        a.a_scale += m0;
        a.Y = (typename elem_of<DT>::type*)a.Y + m0 * a.N;
        a.M = min(a.M - m0, (int64_t)(16 * MG));
    }
    const int M = (int)a.M, K = a.K;
    const int lr = lane >> 3, lp = lane & 7;  // row of 8 and piece that the lane loads
    const int nfull = K / 128;  // whole units; what is left of k is one more, of wave nfull % 8
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NF);
    const auto b_row = [&](int g, int i) { return a.b + min(n0 + 16 * g + 8 * i + lr, a.N - 1) * a.ldb; };
    const auto a_row = [&](int g, int i) { return a.a + (int64_t)min(16 * g + 8 * i + lr, M - 1) * a.lda; };
    u32x4_t w[2][U][NF][2], x[2][U][XG ? XG : 1][2], wt[NF][2], xt[XG ? XG : 1][2];
    // step s: U units of each wave
    constexpr int STEP = U * kFewWaves;
    const auto loads = [&](auto set, int step) __attribute__((always_inline)) {
        static_for<0, U>([&](auto u) {
            const int at = step * STEP + u * kFewWaves + wave;
            if (at < nfull) {
                const int k = at * 128 + lp * 16;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int g = 0; g < NF; ++g) w[set][u][g][i] = *(const u32x4_u1*)(b_row(g, i) + k);
#pragma unroll
                    for (int g = 0; g < XG; ++g) x[set][u][g][i] = *(const u32x4_u1*)(a_row(g, i) + k);
                }
            }
        });
    };
    constexpr std::integral_constant<int, 0> first = {};
    constexpr std::integral_constant<int, 1> second = {};
    const bool tail = K % 128 != 0 && wave == nfull % kFewWaves;
    const auto load_tail = [&]() __attribute__((always_inline)) {
        if (tail) {
            const int k = nfull * 128 + lp * 16, n = max(0, min(16, K - k));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int g = 0; g < NF; ++g) wt[g][i] = bytes16(b_row(g, i) + min(k, K - 1), n);
#pragma unroll
                for (int g = 0; g < XG; ++g) xt[g][i] = bytes16(a_row(g, i) + min(k, K - 1), n);
            }
        }
    };
    // this wave's pieces: [NF + XG][16 rows][8], those of a row in the order piece ^ row
    u32x4_t* own = smem + wave * ((NF + XG) * UNIT);
    // AK >= 0: the rows' int8, [M][kpad / 16] (after what the waves' pieces and sums need)
    u32x4_t* q_s = smem + kFewWaves * (NF * UNIT);
    __shared__ float scale_s[kFewWaves];
    if constexpr (AK >= 0) {
        typedef typename elem_of<AK>::type E;
        constexpr int V = kVec<AK>, KEEP = 4;
        __shared__ uint32_t max_s[kFewWaves];
        // 8 / (M to a power of two) waves a row, KEEP vectors a lane in registers
        const int waves = M == 1 ? 8 : M == 2 ? 4 : M <= 4 ? 2 : 1, row = wave / waves, nl = 64 * waves;
        const int l = (wave % waves) * 64 + lane;
        const E* X = (const E*)f.X + (int64_t)min(row, M - 1) * K;
        u32x4_t keep[KEEP];
        RowMax<AK> largest;
        const auto vec = [&](int c) {
            const int e = (c * nl + l) * V;
            return load16_first(X + min(e, K), max(0, min(V, K - e)));
        };
#pragma unroll
        for (int c = 0; c < KEEP; ++c) keep[c] = vec(c);
        loads(first, 0);
        load_tail();
#pragma unroll
        for (int c = 0; c < KEEP; ++c) largest.add(keep[c]);
        for (int c = KEEP; c * nl * V < K; ++c) largest.add(vec(c));
        uint32_t mx = wave_max_u32(largest.bits());
        if (lane == 0) max_s[wave] = mx;
        __syncthreads();
        // (a row's waves are neighbours: lanes past them look at the first again)
        mx = wave_max_u32(max_s[row * waves + (lane < waves ? lane : 0)]);
        const RowScale rs(mx);
        if (row < M) {
            if (l == 0) scale_s[row] = rs.scale;
            const auto out = [&](int c, u32x4_t v) {
                const int e = (c * nl + l) * V;
                if (e >= f.kpad) return;
                float g[V];
                uint32_t q[V / 4];
                unpack16<AK>(v, g);
                rs.bytes<V>(g, q);
                char* d = (char*)(q_s + row * (f.kpad / 16) + ((e / 16) ^ (row & 7))) + e % 16;
                if constexpr (V == 8) *(u32x2_t*)d = u32x2_t{q[0], q[1]};
                else *(uint32_t*)d = q[0];
            };
#pragma unroll
            for (int c = 0; c < KEEP; ++c) out(c, keep[c]);
            for (int c = KEEP; c * nl * V < f.kpad; ++c) out(c, vec(c));
        }
        __syncthreads();
    } else {
        loads(first, 0);
        load_tail();
    }
    i32x4_t acc[NF][MG] = {};
    const int ir = lane & 15, ip = lane >> 4;  // the operand's row and 16 of 64 k
    const auto mul = [&](const u32x4_t (&w)[NF][2], const u32x4_t (&x)[XG ? XG : 1][2], int u) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = (8 * i + lr) * 8 + (lp ^ lr);
#pragma unroll
            for (int g = 0; g < NF; ++g) own[g * UNIT + at] = w[g][i];
#pragma unroll
            for (int g = 0; g < XG; ++g) own[(NF + g) * UNIT + at] = x[g][i];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = ir * 8 + ((4 * s + ip) ^ (ir & 7));
            u32x4_t fx[MG];
#pragma unroll
            for (int g = 0; g < MG; ++g) {
                if constexpr (AK < 0) fx[g] = own[(NF + g) * UNIT + at];
                else fx[g] = ir < M ? q_s[ir * (f.kpad / 16) + ((u * 8 + 4 * s + ip) ^ (ir & 7))] : u32x4_t{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const u32x4_t fw = own[j * UNIT + at];
#pragma unroll
                for (int g = 0; g < MG; ++g) acc[j][g] = mfma_i8(fw, fx[g], acc[j][g]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    };
    const auto muls = [&](auto set, int step) __attribute__((always_inline)) {
        static_for<0, U>([&](auto u) {
            const int at = step * STEP + u * kFewWaves + wave;
            if (at < nfull) mul(w[set][u], x[set][u], at);
        });
    };
    for (int step = 0; step * STEP < nfull; step += 2) {
        loads(second, step + 1);
        muls(first, step);
        loads(first, step + 2);
        muls(second, step + 1);
    }
    if (tail) mul(wt, xt, nfull);
    // the waves' sums join: [wave][NF][MG][64]
    __syncthreads();
    i32x4_t* red = (i32x4_t*)smem;
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int g = 0; g < MG; ++g) red[((wave * NF + j) * MG + g) * 64 + lane] = acc[j][g];
    __syncthreads();
    for (int o = t; o < NF * MG * 64; o += 64 * kFewWaves) {
        const int l = o & 63, g = (o >> 6) % MG, j = (o >> 6) / MG;
        const int m = 16 * g + (l & 15);
        const int64_t n = n0 + 16 * j + 4 * (l >> 4);
        if (m >= M || n >= a.N) continue;
        i32x4_t sum = red[o];
#pragma unroll
        for (int wv = 1; wv < kFewWaves; ++wv) sum += red[wv * (NF * MG * 64) + o];
        float v[4];
        Columns<DT>(a, n).values(sum, AK < 0 ? a.a_scale[m] : scale_s[AK < 0 ? 0 : m], v);
        store4<DT>(a.Y, m * a.N + n, v, (int)min((int64_t)4, a.N - n));
    }
}

// ------------------------------------------------------------------ tiles
// acc = sum over nk stages of 128 k, two blocks of 64 each, NB stages in LDS
// (row_loop.hpp).  During the first block the second's fragments are read; then the
// barrier that retires the stage and publishes the next; during the second block the
// next stage's first fragments, and the DMA of stage kt + NB.
// KS groups of 4 waves take every KS-th stage each, in LDS of their own.
template <int BT, int NB, int KS, class SA, class SB>
struct Loop8 {
    static constexpr int TM = BT / 32, NM = TM * TM, OPB = BT * 128, STAGE = 2 * OPB, LA = SA::PER_WAVE;
    f32x4_t (&acc)[TM][TM];
    char* smem;
    const SA& sa;
    const SB& sb;
    int nk, lane, wave, group, rowa, rowb;
    u32x4_t fa[2][TM], fb[2][TM];

    __device__ __forceinline__ char* at(int kt) const { return smem + (group * NB + kt % NB) * STAGE; }
    template <int s, int i>
    __device__ __forceinline__ void read(const char* st) {
        if constexpr (i % 2 == 0) fb[s][i / 2] = read_frag16<BT, true>(st + OPB, rowb + 8 * i, s, lane);
        else fa[s][i / 2] = read_frag16<BT, true>(st, rowa + 8 * (i - 1), s, lane);
    }
    template <int d>
    __device__ __forceinline__ void dma(const i32x4_t& ra, const i32x4_t& rb, uint32_t l, int kt) const {
        if constexpr (d < LA) sa.one(ra, l, kt * KS + group, wave, d);
        else sb.one(rb, l + OPB, kt * KS + group, wave, d - LA);
    }
    template <bool Z>
    __device__ __forceinline__ void stage(int kt) {
        const char *st = at(kt), *nx = at(kt + 1);
        phase<3, TM, TM, Z>(acc, fa[0], fb[0], [&](auto xc) {
            spread<NM, 2 * TM, decltype(xc)::value>([&](auto i) { read<1, decltype(i)::value>(st); });
        });
        wait_vm<(NB - 2) * 2 * LA>();  // this wave's DMA of stage kt + 1 has landed
        __syncthreads();               // ... every wave's; and every read of stage kt is done
        fence_sched();
        const int next = (kt + NB) * KS + group;
        const i32x4_t ra = sa.rsrc(next, nk), rb = sb.rsrc(next, nk);
        const uint32_t l = lds_addr(st);
        phase<3, TM, TM, false>(acc, fa[1], fb[1], [&](auto xc) {
            constexpr int x = decltype(xc)::value;
            spread<NM, 2 * LA, x>([&](auto d) { dma<decltype(d)::value>(ra, rb, l, kt + NB); });
            spread<NM, 2 * TM, x>([&](auto i) { read<0, decltype(i)::value>(nx); });
        });
    }
    __device__ __forceinline__ void run() {
        for (int kt = 0; kt < NB; ++kt) {
            const i32x4_t ra = sa.rsrc(kt * KS + group, nk), rb = sb.rsrc(kt * KS + group, nk);
            const uint32_t l = lds_addr(at(kt));
            static_for<0, 2 * LA>([&](auto d) { dma<decltype(d)::value>(ra, rb, l, kt); });
        }
        wait_vm<(NB - 1) * 2 * LA>();
        __syncthreads();
        static_for<0, 2 * TM>([&](auto i) { read<0, decltype(i)::value>(at(0)); });
        stage<true>(0);
        for (int kt = 1; kt * KS < nk; ++kt) stage<false>(kt);
        wait_vm<0>();
        acc_fence(acc);
    }
};

// Results of a wave's H x H block at (wr, wc), from the accumulators' layout
template <int DT, int TM>
__device__ __forceinline__ void tile_store(const ProductArgs& a, const f32x4_t (&acc)[TM][TM], int64_t wr, int64_t wc, int lane) {
    float sa[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = a.a_scale[min(wr + 16 * i + (lane & 15), a.M - 1)];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t n = wc + 16 * j + 4 * (lane >> 4);
        if (n >= a.N) continue;
        const Columns<DT> col(a, n);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = wr + 16 * i + (lane & 15);
            float v[4];
            col.values(__builtin_bit_cast(i32x4_t, acc[i][j]), sa[i], v);
            if (m < a.M) store4<DT>(a.Y, m * a.N + n, v, (int)min((int64_t)4, a.N - n));
        }
    }
}
// ... through LDS of the wave's own (32 rows at a time), by whole rows of 16 bytes a
// lane.  Whole blocks of a Y whose rows are 16-byte aligned.
template <int DT, int TM>
__device__ __forceinline__ void tile_store_rows(const ProductArgs& a, const f32x4_t (&acc)[TM][TM], int64_t wr, int64_t wc,
                                                char* own, int lane) {
    constexpr int H = 16 * TM, EB = DT == 2 ? 4 : 2, W = H * EB, CPR = W / 16, NCH = 32 * CPR / 64, SWZ = CPR < 8 ? CPR - 1 : 7;
    const auto slot = [](int row, int piece) { return (piece ^ (row & SWZ)) << 4; };
#pragma unroll
    for (int h = 0; h < TM / 2; ++h) {
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int g = lane >> 4;
            const Columns<DT> col(a, wc + 16 * j + 4 * g);
#pragma unroll
            for (int ii = 0; ii < 2; ++ii) {
                const int row = 16 * ii + (lane & 15);
                float v[4];
                col.values(__builtin_bit_cast(i32x4_t, acc[2 * h + ii][j]), a.a_scale[wr + 32 * h + row], v);
                const int byte = (16 * j + 4 * g) * EB;
                char* d = own + row * W + slot(row, byte >> 4) + (byte & 15);
                if constexpr (DT == 2) *(f32x4_t*)d = f32x4_t{v[0], v[1], v[2], v[3]};
                else *(u32x2_t*)d = u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
            }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
            const int row = (q * 64 + lane) / CPR, ch = (q * 64 + lane) % CPR;
            *(u32x4_t*)((char*)a.Y + ((wr + 32 * h + row) * a.N + wc) * EB + ch * 16) =
                *(const u32x4_t*)(own + row * W + slot(row, ch));
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// BT x BT tiles, KS groups of 4 waves of (BT / 2)^2, operands of 16-byte aligned rows.
// KT: K is not a multiple of 128; a's pieces past it are zeros, so b's need not be.
template <int BT, int NB, int KS, int DT, bool KT>
__global__ __launch_bounds__(NT * KS, KS * NB * BT * 256 <= 80 * 1024 ? 2 * KS : KS) void int8_tile_kernel(
    ProductArgs a, int tiles_m, int tiles_n) {
    typedef Loop8<BT, NB, KS, RowSrc<BT, KT>, RowSrc<BT, false>> L;
    constexpr int TM = L::TM, H = BT / 2;
    __shared__ __attribute__((aligned(1024))) char smem[KS * NB * L::STAGE];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane((t >> 6) & 3);
    const int group = __builtin_amdgcn_readfirstlane(t >> 8);
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    grouped_order(xcd_remap((int)blockIdx.x, (int)gridDim.x), tiles_m, tiles_n, 4, tm, tn);
    const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
    RowSrc<BT, KT> sa;
    RowSrc<BT, false> sb;
    sa.init(a.a, (uint32_t)a.lda, (uint32_t)a.K, m0, a.M, lane);
    sb.init(a.b, (uint32_t)a.ldb, (uint32_t)a.K, n0, a.N, lane);
    f32x4_t acc[TM][TM];
    L loop{acc, smem, sa, sb, (a.K + 127) / 128, lane, wave, group, wm * H, wn * H};
    loop.run();
    __syncthreads();  // every wave is done with the last stage
    if constexpr (KS > 1) {
        // the groups' sums join (integers: in any order), past what the results need of LDS
        i32x4_t* red = (i32x4_t*)(smem + 4 * 32 * H * 4) + wave * (TM * TM * 64) + lane;
        if (group) {
#pragma unroll
            for (int i = 0; i < TM * TM; ++i)
                red[((group - 1) * 4 * TM * TM + i) * 64] = __builtin_bit_cast(i32x4_t, acc[i / TM][i % TM]);
        }
        __syncthreads();
        if (group) return;
#pragma unroll
        for (int g = 0; g < KS - 1; ++g)
#pragma unroll
            for (int i = 0; i < TM * TM; ++i)
                acc[i / TM][i % TM] = __builtin_bit_cast(
                    f32x4_t, __builtin_bit_cast(i32x4_t, acc[i / TM][i % TM]) + red[(g * 4 * TM * TM + i) * 64]);
    }
    const int64_t wr = m0 + wm * H, wc = n0 + wn * H;
    constexpr int EB = DT == 2 ? 4 : 2;
    if (wr + H <= a.M && wc + H <= a.N && a.N * EB % 16 == 0 && ((uintptr_t)a.Y & 15) == 0)
        tile_store_rows<DT, TM>(a, acc, wr, wc, smem + wave * (32 * H * EB), lane);
    else
        tile_store<DT, TM>(a, acc, wr, wc, lane);
}

// Rows of K bytes at any byte -> rows of ld, a multiple of 16, zeros past K; of up to
// two operands.  A piece is read as the five words around it and shifted into place; by
// 16-byte loads at odd bytes the call takes as long (300 x 2005 x 2048: 15.9 us both; 2000 x
// 2005 x 8192: 53.0, so 53.7).
struct AlignArgs {
    const int8_t* x[2];
    int8_t* y[2];
    int64_t rows[2];
    int64_t ld;
    int K;
};
// A wave takes a row.
__global__ __launch_bounds__(256) void int8_align_kernel(AlignArgs a) {
    const int64_t all = a.rows[0] + a.rows[1];
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < all; r += (int64_t)gridDim.x * 4) {
        const int o = r >= a.rows[0];
        const int64_t row = r - (o ? a.rows[0] : 0);
        const int8_t *x = a.x[o], *from = x + row * a.K, *end = x + a.rows[o] * a.K;
        int8_t* to = a.y[o] + row * a.ld;
        const uint32_t by = (uint32_t)((uintptr_t)from & 3);
        for (int k = (threadIdx.x & 63) * 16; k < a.ld; k += 1024) {
            const int n = a.K - k;
            const int8_t* p = from + k;
            u32x4_t v;
            if (p - by >= x && p + 20 <= end) {
                const uint32_t* w = (const uint32_t*)(p - by);
                const u32x4_t q = *(const u32x4_u4*)w;
                const uint32_t e = w[4];
                v = u32x4_t{__builtin_amdgcn_alignbyte(q.y, q.x, by), __builtin_amdgcn_alignbyte(q.z, q.y, by),
                            __builtin_amdgcn_alignbyte(q.w, q.z, by), __builtin_amdgcn_alignbyte(e, q.w, by)};
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (n < 4 * d + 4) v[d] &= n <= 4 * d ? 0u : (1u << (8 * (n - 4 * d))) - 1u;
            } else {
                v = bytes16(p, n);
            }
            *(u32x4_t*)(to + k) = v;
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

template <int DT, int NF, int MG, int U, int AK>
void few_go(const FewArgs& f, hipStream_t s) {
    constexpr int XG = AK < 0 ? MG : 0;
    const size_t pieces = (size_t)kFewWaves * (NF + XG) * 2048 + (AK < 0 ? 0 : (size_t)f.p.M * f.kpad);
    const size_t lds = std::max(pieces, (size_t)kFewWaves * NF * MG * 1024);
    const dim3 grid((unsigned)((f.p.N + 16 * NF - 1) / (16 * NF)), (unsigned)((f.p.M + 16 * MG - 1) / (16 * MG)));
    log_choice("int8_matmul: %lld rows streamed, %d x %d a workgroup, %d units at once%s", (long long)f.p.M, 16 * MG,
               16 * NF, U, AK < 0 ? "" : ", quantised there");
    int8_few_kernel<DT, NF, MG, U, AK><<<grid, 64 * kFewWaves, lds, s>>>(f);
}
// 16 columns a workgroup while that makes no more of them than there are CUs, or, of
// rows up to 16, two a CU; 32 beyond (us, bf16, graph replays: 1 row, 4096 x 4096
// 6.5 and 7.5, 4096 x 14336 19.2 and 16.9; 43 rows, 4096 x 4104 12.1 and 8.6).  Four
// units of b a wave at once where one round of them is all there is (1 row, 4096 x
// 4096: 6.5, by two 7.5), two where workgroups share a CU (8192 x 8192: 16.6, by four 19.2).
template <int DT, int AK>
void few_columns(const FewArgs& f, hipStream_t s) {
    const int64_t n16 = (f.p.N + 15) / 16;
    if constexpr (AK >= 0) {
        if (n16 <= 512) few_go<DT, 1, 1, 4, AK>(f, s);
        else few_go<DT, 2, 1, 2, AK>(f, s);
    } else if (f.p.M <= 16) {
        if (n16 <= 256) few_go<DT, 1, 1, 4, -1>(f, s);
        else if (n16 <= 512) few_go<DT, 1, 1, 2, -1>(f, s);
        else few_go<DT, 2, 1, 2, -1>(f, s);
    } else if (f.p.M <= 32) {
        if (n16 <= 256) few_go<DT, 1, 2, 2, -1>(f, s);
        else few_go<DT, 2, 2, 1, -1>(f, s);
    } else {
        if (n16 * ((f.p.M + 63) / 64) <= 256) few_go<DT, 1, 4, 1, -1>(f, s);
        else few_go<DT, 2, 4, 1, -1>(f, s);
    }
}

// K = 4096 (32 stages, bf16, us by tiles of 64 / 128 / 256): 256 x 4096 10.7 / 20 / 46, 512 x 4096
// 17 / 20.5 / 47, 2048 x 4096 58 / 36 / 50, 4096 x 4096 107 / 68 / 61, 8192 x 8192 423 /
// 277 / 229; K = 8192: 4096 x 1024 53 / 39 / 81, 4096 x 128 15 / 34 / 79.
constexpr TileTimes kTiles8[] = {{64, 512, 3, 0.2, 0.24, 0.45}, {128, 512, 6, 0.42, 0.45, 0.94},
                                 {256, 256, 14, 0.9, 1.45, 1.45}};
constexpr int kFewRows = 64;

// what is streamed: few rows, or rows that the tiles cannot take (aligned K, but a base on
// an odd byte: 1024 x 4096 x 4096 69 us, where tiles take 23.5).  17 to 64 rows while a
// workgroup of 32 columns each finds a CU of its own, as the tiles are ahead from the
// second turn on (K = 4096, us streamed and by tiles of 64, 17 / 32 / 64 rows: 4096 columns
// 8.3 9.2 / 8.3 8.8 / 8.8 9.6; 8192 10.1 11.4 / 10.5 11.8 / 12.6 13.6; 8208 13.7 12.4 / 13.7 12.7 / 17.5
// 14.2; 14336 17.1 16.0 / 18.3 16.0 / 23.1 17.1; 28672 31 27 / 33 28 / 43 29).
bool streams(const ProductArgs& a, bool aligned) { return !aligned || a.M <= 16 || (a.M <= kFewRows && a.N <= 8192); }

template <int DT>
hipError_t product_run(const ProductArgs& a, hipStream_t s) {
    if (a.K == 0) {
        int8_bias_kernel<DT><<<dim3((unsigned)std::min<int64_t>((a.M * a.N + 255) / 256, 1 << 16)), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    const bool aligned = a.lda % 16 == 0 && a.ldb % 16 == 0 && (((uintptr_t)a.a | (uintptr_t)a.b) & 15) == 0;
    if (streams(a, aligned)) {
        constexpr int64_t kMost = 65535 * kFewRows;  // rows a launch
        for (int64_t m = 0; m < a.M; m += kMost) {
            ProductArgs p = a;
            p.a += m * a.lda;
            p.a_scale += m;
            p.Y = (typename elem_of<DT>::type*)a.Y + m * a.N;
            p.M = std::min(a.M - m, kMost);
            few_columns<DT, -1>({p, nullptr, 0}, s);
        }
        return hipGetLastError();
    }
    const auto count = [&](int bt) { return ((a.M + bt - 1) / bt) * ((a.N + bt - 1) / bt); };
    const int bt = pick_tile(kTiles8, (a.K + 127) / 128, count);
    const int64_t n = count(bt);
    const auto tiles = [&](auto whole, auto ragged, int ks) {
        const int tm = (int)((a.M + bt - 1) / bt), tn = (int)((a.N + bt - 1) / bt);
        log_choice("int8_matmul: %lld x %lld x %d, tiles of %d%s%s", (long long)a.M, (long long)a.N, a.K, bt,
                   ks > 1 ? ", two groups of waves" : "", a.K % 128 ? ", ragged" : "");
        if (a.K % 128 == 0) whole<<<dim3((unsigned)n), NT * ks, 0, s>>>(a, tm, tn);
        else ragged<<<dim3((unsigned)n), NT * ks, 0, s>>>(a, tm, tn);
    };
    // where every tile has a CU of its own, two groups of waves take turns at the
    // stages (1024 x 4096 x 4096: 25.9 -> 23.6 us)
    if (bt == 64 && n <= 256) tiles(int8_tile_kernel<64, 4, 2, DT, false>, int8_tile_kernel<64, 4, 2, DT, true>, 2);
    else if (bt == 64) tiles(int8_tile_kernel<64, 4, 1, DT, false>, int8_tile_kernel<64, 4, 1, DT, true>, 1);
    else if (bt == 128 && n <= 256) tiles(int8_tile_kernel<128, 2, 2, DT, false>, int8_tile_kernel<128, 2, 2, DT, true>, 2);
    else if (bt == 128) tiles(int8_tile_kernel<128, 2, 1, DT, false>, int8_tile_kernel<128, 2, 1, DT, true>, 1);
    else tiles(int8_tile_kernel<256, 2, 1, DT, false>, int8_tile_kernel<256, 2, 1, DT, true>, 1);
    return hipGetLastError();
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t padded(int64_t K) { return (K + 15) / 16 * 16; }

}  // namespace

hipError_t launch_quantize_rows(const void* X, int8_t* Q, float* scale, int64_t M, int64_t K, int dt, hipStream_t s) {
    return quantise_dt({X, Q, scale, M, K, (int)K}, dt, s);
}

// Operands whose K is no multiple of 16 are copied to rows that are, where the tiles will
// take them.  They are streamed up to 128 rows (100 x 2005 x 8192: 17.1 us, copied
// 19.4) and where every CU has one workgroup of 64 rows and 32 columns at most (300 x 2005 x
// 512: 7.6 and 11.9); beyond, streaming b for every 64 rows costs more (300 x 2005 x 8192:
// 38 and 27).
bool copies(int64_t M, int64_t K, int64_t N) {
    return K % 16 && M > 128 && (M + 63) / 64 * ((N + 31) / 32) > 256;
}

size_t int8_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N, bool quantise) {
    const size_t ld = (size_t)padded(K), copy = copies(M, K, N);
    return (quantise ? align256((size_t)M * 4) : 0) + (quantise || copy ? align256((size_t)M * ld) : 0) +
           (copy ? align256((size_t)N * ld) : 0);
}

hipError_t launch_int8_matmul(const Int8Args& x, int dt, void* ws, hipStream_t s) {
    ProductArgs a = {(const int8_t*)x.a, (const int8_t*)x.b, x.a_scale, x.b_scale, x.bias, x.Y, x.M, x.N, x.K, x.K, (int)x.K};
    // one or two rows, which every workgroup of the product quantises for itself: 8.7 us for
    // 1 row of 4096 x 4096, with a kernel before it 9.3 (8 rows: 12.8 and 9.4)
    const int64_t kpad = (x.K + 127) / 128 * 128;
    if (x.a_kind == dt && x.K > 0 && x.M <= 2 && kpad <= 16384) {
        const FewArgs f = {a, x.a, (int)kpad};
        if (dt == 0) few_columns<0, 0>(f, s);
        else if (dt == 1) few_columns<1, 1>(f, s);
        else few_columns<2, 2>(f, s);
        return hipGetLastError();
    }
    const int64_t ld = padded(x.K);
    const bool copy = copies(x.M, x.K, x.N);
    char* w = (char*)ws;
    AlignArgs al = {};
    al.ld = ld;
    al.K = (int)x.K;
    if (x.a_kind >= 0) {
        float* scale = (float*)w;
        w += align256((size_t)x.M * 4);
        const hipError_t e = quantise_dt({x.a, (int8_t*)w, scale, x.M, ld, (int)x.K}, x.a_kind, s);
        if (e != hipSuccess) return e;
        a.a = (int8_t*)w;
        a.lda = ld;
        a.a_scale = scale;
        w += align256((size_t)x.M * ld);
    } else if (copy) {
        al.x[0] = a.a;
        al.y[0] = (int8_t*)w;
        al.rows[0] = x.M;
        a.a = (int8_t*)w;
        a.lda = ld;
        w += align256((size_t)x.M * ld);
    }
    if (copy) {
        al.x[1] = a.b;
        al.y[1] = (int8_t*)w;
        al.rows[1] = x.N;
        a.b = (int8_t*)w;
        a.ldb = ld;
        int8_align_kernel<<<(unsigned)std::min<int64_t>((al.rows[0] + al.rows[1] + 3) / 4, 1 << 16), 256, 0, s>>>(al);
    }
    return dt == 0 ? product_run<0>(a, s) : dt == 1 ? product_run<1>(a, s) : product_run<2>(a, s);
}

}  // namespace omm
