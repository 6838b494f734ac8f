// The router in training: per-expert counts with the balance and z losses, and
// the gradient of everything that reads the router's logits.
//
//   p = softmax(logits[m]) over E experts, lse[m] its log-sum-exp; n tokens counted
//   counts[e] = number of selections of e by those tokens,  f = counts / sum counts
//   losses = ( E sum_e f[e] mean_m p[m, e],  mean_m lse[m]^2 )
//   d logits = g0 E / n p (f - sum f p) + g1 2 / n lse p + what the selections' weights get:
//     not renormalised  p (G - sum p G),          G[e] = sum of the gradients of e's selections
//     renormalised      p / D (G - c sum p G / D), c[e] = selections of e, D = sum p c
//
// Each is one read of the logits (and one write): 16384 tokens of 64 experts are 2 to
// 4 MB, so launches and the join of the workgroups' sums are the time (8.4 us for counts
// and losses, 6.3 for the gradient).  Where there is more, the instructions of a logit
// are: 40709 tokens of 160 experts, fp32, 26 MB, take 17 us and 17.8 (2.9 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kernels.hpp"
#include "row_select.hpp"

namespace omm {

namespace {

constexpr int kMaxE = 512;

__device__ __forceinline__ float row16_maxf(float v) {
    v = fmaxf(v, __uint_as_float(dpp_u32<0x128, 0xf>(0u, __float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp_u32<0x124, 0xf>(0u, __float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp_u32<0x122, 0xf>(0u, __float_as_uint(v))));
    return fmaxf(v, __uint_as_float(dpp_u32<0x121, 0xf>(0u, __float_as_uint(v))));
}

// 16 lanes a token (as in the routing).  Lane l holds NE experts: with four of each 64 in
// a row (of each 16 one where E <= 16), a wave reads whole lines of a wide router.
template <int NE>
struct Layout {
    static constexpr int W = NE < 4 ? 1 : 4;
    static __device__ __forceinline__ constexpr int at(int l, int i) { return (i / W) * (16 * W) + l * W + i % W; }
};
// rows that can be read and written in fours
template <int DT>
__device__ __forceinline__ bool whole_fours(const void* p, int E) {
    return E % 4 == 0 && (uintptr_t)p % (4 * sizeof(typename elem_of<DT>::type)) == 0;
}
// A token's logits as they are stored; every load is on its way before the first is used.
template <int DT, int NE>
struct Row {
    typedef typename elem_of<DT>::type T;
    typedef Layout<NE> L;
    typedef T TW __attribute__((ext_vector_type(L::W)));
    TW v[NE / L::W];
    __device__ __forceinline__ void load(const void* logits, int64_t m, int E, int l, bool wide) {
        const T none = f32_elem<DT>(-__builtin_inff());
        const T* row = (const T*)logits + m * E;
#pragma unroll
        for (int i = 0; i < NE; i += L::W) v[i / L::W] = none;
        if (L::W == 4 && wide) {
#pragma unroll
            for (int i = 0; i < NE; i += 4)
                if (i < inside() || L::at(l, i) < E) v[i / L::W] = *(const TW*)(row + L::at(l, i));
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (i < inside() || L::at(l, i) < E) v[i / L::W][i % L::W] = row[L::at(l, i)];
        }
    }
    __device__ __forceinline__ void get(float (&x)[NE]) const {
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = elem_f32<DT>(v[i / L::W][i % L::W]);
    }
    // experts of a lane that this layout is not chosen without (see for_experts)
    static __device__ __forceinline__ constexpr int inside() { return NE <= 4 ? 0 : NE <= 16 ? NE - 4 : NE - 8; }
};
// exp(x) for x <= 0 (a NaN stays one): 2^t by the exponential unit and what t = x log2(e)
// was rounded by, to first order; below 2^-126 it is 0, nothing in a sum of 1 and more.
// The library's takes twice the instructions (the gradient of 40709 tokens of 512 experts,
// bf16: 45 us, so 41).
__device__ __forceinline__ float exp_small(float x) {
    constexpr float kHigh = 1.44269504f, kLow = 1.92596299e-8f;  // log2(e) = kHigh + kLow
    x = x < -150.0f ? -150.0f : x;
    const float t = x * kHigh, y = __builtin_amdgcn_exp2f(t);
    return fmaf(y, (fmaf(x, kHigh, -t) + x * kLow) * 0.693147181f, y);
}
// logits -> probabilities; returns the log-sum-exp.  A row of nothing but -inf
// has probabilities and log-sum-exp 0; one with a NaN or +inf has NaN.
template <int NE>
__device__ __forceinline__ float softmax16(float (&x)[NE]) {
    float mx = x[0], s = 0.0f;
#pragma unroll
    for (int i = 1; i < NE; ++i) mx = fmaxf(mx, x[i]);
    mx = row16_maxf(mx);
    if (mx == -__builtin_inff()) mx = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        x[i] = exp_small(x[i] - mx);
        s += x[i];
    }
    s = row16_sum(s);
    const float r = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] *= r;
    return s == 0.0f ? 0.0f : mx + logf(s);
}

__device__ __forceinline__ int64_t index_of(const void* ids, int64_t i, int idx64) {
    return idx64 ? ((const int64_t*)ids)[i] : (int64_t)((const int32_t*)ids)[i];
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}
__device__ __forceinline__ int wave_sum_int(int v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// ------------------------------------------------------------------ counts and losses
// A workgroup's share: probabilities and counts by expert, and (sum lse^2, tokens);
// then what the join's workgroups hand to the last of them.
struct Parts {
    double* dot;     // [join workgroup]: sum of p counts
    int64_t* total;  // [join workgroup]: sum of counts
    uint32_t* done;  // join workgroups that are
    float* p;        // [block][E]
    int32_t* count;  // [block][E]
    float* z;        // [block]
    int32_t* n;      // [block]
};
constexpr int kJoinE = 64, kMaxJoin = kMaxE / kJoinE;  // experts of a join workgroup
constexpr int kHead = kMaxJoin * 16 + 16;              // bytes before p
__host__ __device__ inline Parts parts_of(void* ws, int blocks, int E) {
    Parts r;
    r.dot = (double*)ws;
    r.total = (int64_t*)(r.dot + kMaxJoin);
    r.done = (uint32_t*)(r.total + kMaxJoin);
    r.p = (float*)((char*)ws + kHead);
    r.count = (int32_t*)(r.p + (int64_t)blocks * E);
    r.z = (float*)(r.count + (int64_t)blocks * E);
    r.n = (int32_t*)(r.z + blocks);
    return r;
}

// One workgroup's tokens: sums of its probabilities psum[wave][e], counts, lse^2 and tokens in LDS
template <int DT, int NE, int NW>
struct BalanceBlock {
    int32_t count[kMaxE];
    float psum[NW][16 * NE];
    float zsum[4 * NW];
    int32_t nsum[4 * NW];
    __device__ __forceinline__ void run(const MoeBalanceArgs& a) {
        const int t = threadIdx.x, l = t & 15, E = (int)a.E;
        for (int e = t; e < E; e += 64 * NW) count[e] = 0;
        __syncthreads();
        float p[NE] = {}, z = 0.0f;
        int n = 0;
        const bool wide = whole_fours<DT>(a.logits, E);
        constexpr int PER = 4 * NW;  // tokens at a time
        const int64_t step = (int64_t)gridDim.x * PER;
        int64_t m = (int64_t)blockIdx.x * PER + (t >> 4);
        Row<DT, NE> row;
        int64_t id = -1;
        bool keep = false;
        const auto load = [&] {
            const int64_t at = m < a.M ? m : a.M - 1;
            keep = m < a.M && (!a.mask || a.mask[at]);
            row.load(a.logits, at, E, l, wide);
            id = l < a.k ? index_of(a.ids, at * a.k + l, a.ids64) : -1;
            m += step;
        };
        if ((int64_t)blockIdx.x * PER < a.M) load();  // (no token: no row to read)
        for (int64_t m0 = (int64_t)blockIdx.x * PER; m0 < a.M; m0 += step) {
            float x[NE];
            row.get(x);
            const bool counts = keep;
            if (keep && id >= 0 && id < E) atomicAdd(&count[id], 1);  // (whole numbers: any order)
            if (m0 + step < a.M) load();
            const float lse = softmax16(x);
            if (counts) {
#pragma unroll
                for (int i = 0; i < NE; ++i) p[i] += x[i];
                z += lse * lse;
                ++n;
            }
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            p[i] += __shfl_xor(p[i], 16, 64);
            p[i] += __shfl_xor(p[i], 32, 64);
            if ((t & 63) < 16) psum[t >> 6][Layout<NE>::at(l, i)] = p[i];
        }
        if (l == 0) {
            zsum[t >> 4] = z;
            nsum[t >> 4] = n;
        }
        __syncthreads();
    }
    __device__ __forceinline__ float prob(int e) const {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) p += psum[w][e];
        return p;
    }
};

__device__ __forceinline__ void balance_result(const MoeBalanceArgs& a, double dot, double total, double z, int n) {
    // no token counted: both losses 0; no selection: the balance loss
    a.losses[0] = n && total > 0.0 ? (float)((double)a.E * (dot / total) / n) : 0.0f;
    a.losses[1] = n ? (float)(z / n) : 0.0f;
    a.tokens[0] = n;
}

template <int DT, int NE>
__global__ __launch_bounds__(1024) void balance_parts_kernel(MoeBalanceArgs a, void* ws) {
    __shared__ BalanceBlock<DT, NE, 16> b;
    b.run(a);
    const int t = threadIdx.x, E = (int)a.E;
    const Parts out = parts_of(ws, (int)gridDim.x, E);
    if (t < E) {
        out.p[(int64_t)blockIdx.x * E + t] = b.prob(t);
        out.count[(int64_t)blockIdx.x * E + t] = b.count[t];
    }
    if (t < 64) {
        const float zs = wave_sum(b.zsum[t]);
        const int ns = wave_sum_int(b.nsum[t]);
        if (t == 0) {
            out.z[blockIdx.x] = zs;
            out.n[blockIdx.x] = ns;
            if (blockIdx.x == 0) *out.done = 0;
        }
    }
}

// The join: a workgroup takes 64 experts, thread t expert t % 64 of the parts t / 64,
// t / 64 + 16 ..; up to 64 experts that is all, else the last workgroup to be done sums
// what all of them left (in their order).
__global__ __launch_bounds__(1024) void balance_join_kernel(MoeBalanceArgs a, void* ws, int blocks) {
    __shared__ double ps[16][65];
    __shared__ int32_t cs[16][65];
    __shared__ float zs[16];
    __shared__ int32_t ns[16];
    __shared__ int last;
    const int t = threadIdx.x, E = (int)a.E, e = blockIdx.x * kJoinE + (t & 63), g = t >> 6;
    const Parts in = parts_of(ws, blocks, E);
    const bool first = blockIdx.x == 0;
    const float zt = first && t < blocks ? in.z[t] : 0.0f;
    const int nt = first && t < blocks ? in.n[t] : 0;
    double p = 0.0;
    int32_t c = 0;
    if (e < E) {
#pragma unroll 8
        for (int b = g; b < blocks; b += 16) {
            p += in.p[(int64_t)b * E + e];
            c += in.count[(int64_t)b * E + e];
        }
    }
    ps[g][t & 63] = p;
    cs[g][t & 63] = c;
    const float zw = wave_sum(zt);
    const int nw = wave_sum_int(nt);
    if ((t & 63) == 0) {
        zs[g] = zw;
        ns[g] = nw;
    }
    __syncthreads();
    if (t < 64) {
        p = 0.0;
        c = 0;
        double z = 0.0;
        int n = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            p += ps[k][t];
            c += cs[k][t];
            z += zs[k];
            n += ns[k];
        }
        if (e < E) a.counts[e] = c;
        const double dot = wave_sum64(e < E ? p * c : 0.0), total = wave_sum64(e < E ? (double)c : 0.0);
        if (t == 0) {
            if (gridDim.x == 1) {
                balance_result(a, dot, total, z, n);
            } else {
                __hip_atomic_store(&in.dot[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                __hip_atomic_store(&in.total[blockIdx.x], (int64_t)total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                last = __hip_atomic_fetch_add(in.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
            }
        }
    }
    if (gridDim.x == 1) return;
    __syncthreads();
    if (!last || t >= 64) return;
    // every workgroup of experts, and the parts' (lse^2, tokens)
    const bool in_grid = t < (int)gridDim.x;
    const double dot = wave_sum64(in_grid ? __hip_atomic_load(&in.dot[t], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0);
    const double total = wave_sum64(
        in_grid ? (double)__hip_atomic_load(&in.total[t], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0);
    double z = 0.0;
    int n = 0;
    for (int b = t; b < blocks; b += 64) {
        z += in.z[b];
        n += in.n[b];
    }
    z = wave_sum64(z);
    n = wave_sum_int(n);
    if (t == 0) balance_result(a, dot, total, z, n);
}

// Few tokens: all of it in one workgroup of 16 waves, 64 tokens at a time (a second
// kernel costs 3 to 4 us).
template <int DT, int NE>
__global__ __launch_bounds__(1024) void balance_few_kernel(MoeBalanceArgs a) {
    __shared__ BalanceBlock<DT, NE, 16> b;
    __shared__ double red[16][2];
    b.run(a);
    const int t = threadIdx.x, E = (int)a.E;
    double dot = 0.0, total = 0.0;
    if (t < E) {
        const int c = b.count[t];
        a.counts[t] = c;
        dot = (double)b.prob(t) * c;
        total = c;
    }
    dot = wave_sum64(dot);
    total = wave_sum64(total);
    if ((t & 63) == 0) {
        red[t >> 6][0] = dot;
        red[t >> 6][1] = total;
    }
    __syncthreads();
    if (t >= 64) return;
    const double z = wave_sum64(b.zsum[t]);
    const int n = wave_sum_int(b.nsum[t]);
    dot = wave_sum64(t < 16 ? red[t][0] : 0.0);
    total = wave_sum64(t < 16 ? red[t][1] : 0.0);
    if (t == 0) balance_result(a, dot, total, z, n);
}
constexpr int kFewTokens = 256;

// Workgroups for n turns of a workgroup's tokens, at most `most` and with as many turns each
int64_t even_blocks(int64_t n, int64_t most) {
    const int64_t turns = (n + most - 1) / most;
    return (n + turns - 1) / turns;
}
// Workgroups of the first kernel, which take 64 tokens at a time.  No more than 256, as
// a join workgroup reads 64 experts of each (16384 tokens: 512 parts of 16 tokens a
// turn took the join 14.7 us, 256 KB at the rate of one CU; 40709 tokens of 512 experts:
// 34 us with 128 parts, 27.5 with 256).
int balance_blocks(int64_t M) { return (int)even_blocks((M + 63) / 64, 256); }

// one of the layouts, f(integral_constant): 64 experts a step of 4
template <class F>
void for_experts(int64_t E, const F& f) {
    if (E <= 16) f(std::integral_constant<int, 1>());
    else if (E <= 64) f(std::integral_constant<int, 4>());
    else if (E <= 128) f(std::integral_constant<int, 8>());
    else if (E <= 192) f(std::integral_constant<int, 12>());
    else if (E <= 256) f(std::integral_constant<int, 16>());
    else if (E <= 384) f(std::integral_constant<int, 24>());
    else f(std::integral_constant<int, 32>());
}

template <int DT, int NE>
void balance_go(const MoeBalanceArgs& a, void* ws, hipStream_t s) {
    if (a.M <= kFewTokens) {
        balance_few_kernel<DT, NE><<<1, 1024, 0, s>>>(a);
        return;
    }
    const int blocks = balance_blocks(a.M);
    balance_parts_kernel<DT, NE><<<blocks, 1024, 0, s>>>(a, ws);
    balance_join_kernel<<<(unsigned)((a.E + kJoinE - 1) / kJoinE), 1024, 0, s>>>(a, ws, blocks);
}
template <int DT>
hipError_t balance(const MoeBalanceArgs& a, void* ws, hipStream_t s) {
    for_experts(a.E, [&](auto ne) { balance_go<DT, decltype(ne)::value>(a, ws, s); });
    return hipGetLastError();
}

// ------------------------------------------------------------------ gradient
// value of lane s of 16 neighbouring ones (a DPP row broadcast)
template <int s>
__device__ __forceinline__ uint32_t row16_lane(uint32_t v) { return dpp_u32<0x150 + s, 0xf>(0u, v); }

// g[i], sel[i]: the gradients of expert i's selections and how many there are, every
// selection against the lane's experts
template <int DT, int NE, int s>
__device__ __forceinline__ void select(int id, float gs, int k, int l, float (&g)[NE], float (&sel)[NE]) {
    if (s < k) {  // (uniform)
        const int e = (int)row16_lane<s>((uint32_t)id) - Layout<NE>::at(l, 0);
        const float v = __uint_as_float(row16_lane<s>(__float_as_uint(gs)));
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            g[i] += e == i ? v : 0.0f;
            sel[i] += e == i ? 1.0f : 0.0f;
        }
    }
    if constexpr (s + 1 < 16) select<DT, NE, s + 1>(id, gs, k, l, g, sel);
}
// For many experts that is too much: lane s of a token sums what has its selection's
// expert, and the first of those lanes leaves the sum in the token's row of LDS.
template <int s>
__device__ __forceinline__ void gather_same(int id, float gs, int k, int l, float& g, int& n, bool& first) {
    if (s < k) {
        const bool same = (int)row16_lane<s>((uint32_t)id) == id;
        const float v = __uint_as_float(row16_lane<s>(__float_as_uint(gs)));
        g += same ? v : 0.0f;
        n += same ? 1 : 0;
        if (same && s < l) first = false;
    }
    if constexpr (s + 1 < 16) gather_same<s + 1>(id, gs, k, l, g, n, first);
}
// a wave's writes to LDS, for its other lanes to read
__device__ __forceinline__ void wave_lds() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Selections need not be a token's largest logits (groups, random second choices).  Where
// their probabilities add up to less than this, some may be below fp32's range: their
// weights are then computed among themselves, lane s that of selection s.  Above it, what
// has no probability in fp32 has less than 2^-66 of the weight.
constexpr float kFarBelow = 0x1p-60f;

template <int DT, int NE>
__global__ __launch_bounds__(256) void route_grad_kernel(MoeRouteGradArgs a) {
    typedef typename elem_of<DT>::type T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef Layout<NE> L;
    constexpr bool ROWS = NE > 4;  // selections through rows of LDS, which are zero between two tokens
    __shared__ int32_t count[16 * NE];
    __shared__ float wsum[4];
    __shared__ float grow[ROWS ? 16 : 1][ROWS ? 16 * NE : 1];
    __shared__ uint32_t crow[ROWS ? 16 : 1][ROWS ? 4 * NE : 1];  // a byte an expert
    const int t = threadIdx.x, l = t & 15, E = (int)a.E, k = a.k;
    const bool wide = whole_fours<DT>(a.logits, E) && whole_fours<DT>(a.dlogits, E);
    float f[NE] = {}, cz = 0.0f;
    // what the first token needs is asked for before the counts are summed
    int64_t m = (int64_t)blockIdx.x * 16 + (t >> 4);
    const int64_t step = (int64_t)gridDim.x * 16;
    Row<DT, NE> row;
    float gs = 0.0f;
    int id = -1;
    bool keep = false;
    const auto load = [&] {
        const int64_t at = m < a.M ? m : a.M - 1;
        keep = m < a.M && (!a.mask || a.mask[at]);
        row.load(a.logits, at, E, l, wide);
        id = -1;
        gs = 0.0f;
        if (a.g_weights && l < k) {
            const int64_t i = index_of(a.ids, at * k + l, a.ids64);
            const float v = a.g_weights[at * k + l];
            if (keep && i >= 0 && i < E) {
                id = (int)i;
                gs = v;
            }
        }
    };
    load();
    float* gr = grow[ROWS ? t >> 4 : 0];
    uint32_t* cr = crow[ROWS ? t >> 4 : 0];
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < NE; ++i) gr[i * 16 + l] = 0.0f;
#pragma unroll
        for (int i = 0; i < NE / 4; ++i) cr[i * 16 + l] = 0;
        wave_lds();
    }
    if (a.g_losses) {
        // in fp32, as the counts of several processes may add up to more than int32 holds (exact up to 2^24)
        float c = 0.0f;
        for (int e = t; e < 16 * NE; e += 256) {
            const int v = e < E ? a.counts[e] : 0;
            count[e] = v;
            c += (float)v;
        }
        c = wave_sum(c);
        if ((t & 63) == 0) wsum[t >> 6] = c;
        const int n = a.tokens[0];
        const float g0 = a.g_losses[0], g1 = a.g_losses[1];
        __syncthreads();
        const float total = (wsum[0] + wsum[1]) + (wsum[2] + wsum[3]);
        const float cb = n > 0 && total > 0.0f ? g0 * (float)E / (float)n : 0.0f;
        cz = n > 0 ? g1 * 2.0f / (float)n : 0.0f;
        // f of the formula with its factor
#pragma unroll
        for (int i = 0; i < NE; ++i) f[i] = total > 0.0f ? cb * ((float)count[L::at(l, i)] / total) : 0.0f;
    }
    for (int64_t m0 = (int64_t)blockIdx.x * 16; m0 < a.M; m0 += step) {
        float g[NE] = {}, sel[NE] = {};
        if (a.g_weights) {
            if constexpr (ROWS) {
                float sum = 0.0f;
                int n = 0;
                bool first = id >= 0;
                gather_same<0>(id, gs, k, l, sum, n, first);
                if (first) {
                    gr[id] = sum;
                    ((uint8_t*)cr)[id] = (uint8_t)n;
                }
                wave_lds();
#pragma unroll
                for (int i = 0; i < NE; i += 4) {
                    const f32x4_t v = *(const f32x4_t*)(gr + L::at(l, i));
                    const uint32_t c = cr[L::at(l, i) / 4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[i + j] = v[j];
                        sel[i + j] = (float)(c >> (8 * j) & 0xff);
                    }
                }
                wave_lds();
                if (first) {
                    gr[id] = 0.0f;
                    ((uint8_t*)cr)[id] = 0;
                }
            } else {
                select<DT, NE, 0>(id, gs, k, l, g, sel);
            }
        }
        float x[NE];
        row.get(x);
        const float lse = softmax16(x);  // x: the probabilities
        float pf = 0.0f, pg = 0.0f, pc = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            pf += x[i] * f[i];
            pg += x[i] * g[i];
            pc += x[i] * sel[i];
        }
        pf = row16_sum(pf);
        pg = row16_sum(pg);
        pc = row16_sum(pc);
        const bool far = a.renorm && a.g_weights && keep && pc < kFarBelow;
        const float r = a.renorm ? (pc < kFarBelow ? 0.0f : 1.0f / pc) : 1.0f, mean = pg * r, zl = cz * lse - pf;
        float d[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float w = a.renorm ? r * (g[i] - sel[i] * mean) : g[i] - mean;
            d[i] = keep ? x[i] * (f[i] + zl + w) : 0.0f;
        }
        if (far) {
            // (read once more: nothing but a bit is carried this far for what hardly ever is)
            const int64_t i = l < k ? index_of(a.ids, m * k + l, a.ids64) : -1;
            const bool in = i >= 0 && i < E;
            const float v = in ? a.g_weights[m * k + l] : 0.0f;
            const float y = in ? elem_f32<DT>(((const T*)a.logits)[m * E + i]) : -__builtin_inff();
            float mx = row16_maxf(y);
            if (mx == -__builtin_inff()) mx = 0.0f;
            const float q = exp_small(y - mx), qc = row16_sum(q), w = qc == 0.0f ? 0.0f : q / qc;
            const float term = w * (v - row16_sum(w * v));
            for (int s = 0; s < k; ++s) {
                const int e = __shfl(in ? (int)i : -1, s, 16) - L::at(l, 0);
                const float ts = __shfl(term, s, 16);
#pragma unroll
                for (int c = 0; c < NE; ++c) d[c] += e == L::at(0, c) ? ts : 0.0f;
            }
        }
        const int64_t at = m;
        m += step;
        if (m0 + step < a.M) load();
        if (at < a.M) {
            T* out = (T*)a.dlogits + at * E;
            if (L::W == 4 && wide) {
#pragma unroll
                for (int i = 0; i < NE; i += 4) {
                    T4 v;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = f32_elem<DT>(d[i + j]);
                    if (L::at(l, i) < E) *(T4*)(out + L::at(l, i)) = v;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    if (L::at(l, i) < E) out[L::at(l, i)] = f32_elem<DT>(d[i]);
            }
        }
    }
}

template <int DT>
void route_grad(const MoeRouteGradArgs& a, hipStream_t s) {
    // 5 workgroups a CU are there at a time with 160 experts (40709 tokens: 20.0 us with up
    // to 2048 workgroups, 18.5 with as many turns in each)
    const unsigned blocks = (unsigned)even_blocks((a.M + 15) / 16, 1280);
    for_experts(a.E, [&](auto ne) { route_grad_kernel<DT, decltype(ne)::value><<<blocks, 256, 0, s>>>(a); });
}

}  // namespace

size_t moe_balance_workspace_bytes(int64_t M, int64_t E) {
    return M <= kFewTokens ? 0 : (size_t)kHead + (size_t)balance_blocks(M) * (size_t)(8 * E + 8);
}

hipError_t launch_moe_balance(const MoeBalanceArgs& a, int dt, void* ws, hipStream_t s) {
    return dt == 0 ? balance<0>(a, ws, s) : dt == 1 ? balance<1>(a, ws, s) : balance<2>(a, ws, s);
}

hipError_t launch_moe_route_grad(const MoeRouteGradArgs& a, int dt, hipStream_t s) {
    if (dt == 0) route_grad<0>(a, s);
    else if (dt == 1) route_grad<1>(a, s);
    else route_grad<2>(a, s);
    return hipGetLastError();
}

}  // namespace omm
