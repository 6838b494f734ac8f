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
// Each is one read of the logits (and one write): 16384 tokens of 64 experts are
// 2 MB, so launches and the join of the workgroups' sums are the time.
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// 16 lanes a token (as in the routing): lane l holds experts NE l .. + NE - 1.
template <int DT, int NE>
__device__ __forceinline__ void load_row(const void* logits, int64_t m, int E, int l, float (&x)[NE]) {
    const typename elem_of<DT>::type* row = (const typename elem_of<DT>::type*)logits + m * E;
    if (E == 16 * NE) {
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = elem_f32<DT>(row[l * NE + i]);
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = l * NE + i < E ? elem_f32<DT>(row[l * NE + i]) : -__builtin_inff();
    }
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
        x[i] = expf(x[i] - mx);
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
        constexpr int PER = 4 * NW;  // tokens at a time
        for (int64_t m0 = (int64_t)blockIdx.x * PER; m0 < a.M; m0 += (int64_t)gridDim.x * PER) {
            const int64_t m = m0 + (t >> 4);
            const bool keep = m < a.M && (!a.mask || a.mask[m]);
            float x[NE];
            load_row<DT, NE>(a.logits, m < a.M ? m : a.M - 1, E, l, x);
            const int64_t id = keep && l < a.k ? index_of(a.ids, m * a.k + l, a.ids64) : -1;
            if (id >= 0 && id < E) atomicAdd(&count[id], 1);  // (whole numbers: any order)
            const float lse = softmax16(x);
            if (keep) {
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
            if ((t & 63) < 16) psum[t >> 6][l * NE + i] = p[i];
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

// Workgroups of the first kernel, which take 64 tokens at a time.  No more than 128, as
// a join workgroup reads 64 experts of each (16384 tokens: 512 parts of 16 tokens a
// turn took the join 14.7 us, 256 KB at the rate of one CU).
int balance_blocks(int64_t M) {
    const int64_t n = (M + 63) / 64;
    return (int)(n < 128 ? n : 128);
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
    if (a.E <= 16) balance_go<DT, 1>(a, ws, s);
    else if (a.E <= 64) balance_go<DT, 4>(a, ws, s);
    else if (a.E <= 128) balance_go<DT, 8>(a, ws, s);
    else if (a.E <= 256) balance_go<DT, 16>(a, ws, s);
    else balance_go<DT, 32>(a, ws, s);
    return hipGetLastError();
}

// ------------------------------------------------------------------ gradient
// value of lane s of 16 neighbouring ones (a DPP row broadcast)
template <int s>
__device__ __forceinline__ uint32_t row16_lane(uint32_t v) { return dpp_u32<0x150 + s, 0xf>(0u, v); }

template <int DT, int NE, int s>
__device__ __forceinline__ void select(int id, float gs, int k, int l, float (&g)[NE], float (&sel)[NE]) {
    if (s < k) {  // (uniform)
        const int e = (int)row16_lane<s>((uint32_t)id) - l * NE;
        const float v = __uint_as_float(row16_lane<s>(__float_as_uint(gs)));
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            g[i] += e == i ? v : 0.0f;
            sel[i] += e == i ? 1.0f : 0.0f;
        }
    }
    if constexpr (s + 1 < 16) select<DT, NE, s + 1>(id, gs, k, l, g, sel);
}

template <int DT, int NE>
__global__ __launch_bounds__(256) void route_grad_kernel(MoeRouteGradArgs a) {
    typedef typename elem_of<DT>::type T;
    __shared__ int32_t count[16 * NE];
    __shared__ int32_t wsum[4];
    const int t = threadIdx.x, l = t & 15, E = (int)a.E, k = a.k;
    float f[NE] = {}, cz = 0.0f;
    // what the first token needs is asked for before the counts are summed
    int64_t m = (int64_t)blockIdx.x * 16 + (t >> 4);
    const int64_t step = (int64_t)gridDim.x * 16;
    float x[NE], gs = 0.0f;
    int id = -1;
    bool keep = false;
    const auto load = [&] {
        const int64_t at = m < a.M ? m : a.M - 1;
        keep = m < a.M && (!a.mask || a.mask[at]);
        load_row<DT, NE>(a.logits, at, E, l, x);
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
    if (a.g_losses) {
        int c = 0;
        for (int e = t; e < 16 * NE; e += 256) {
            const int v = e < E ? a.counts[e] : 0;
            count[e] = v;
            c += v;
        }
        c = wave_sum_int(c);
        if ((t & 63) == 0) wsum[t >> 6] = c;
        const int n = a.tokens[0];
        const float g0 = a.g_losses[0], g1 = a.g_losses[1];
        __syncthreads();
        const int total = wsum[0] + wsum[1] + wsum[2] + wsum[3];
        const float cb = n > 0 && total > 0 ? g0 * (float)E / (float)n : 0.0f;
        cz = n > 0 ? g1 * 2.0f / (float)n : 0.0f;
        // f of the formula with its factor
#pragma unroll
        for (int i = 0; i < NE; ++i) f[i] = total > 0 ? cb * ((float)count[l * NE + i] / (float)total) : 0.0f;
    }
    for (int64_t m0 = (int64_t)blockIdx.x * 16; m0 < a.M; m0 += step) {
        float g[NE] = {}, sel[NE] = {};
        if (a.g_weights) select<DT, NE, 0>(id, gs, k, l, g, sel);
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
        const float r = a.renorm ? (pc == 0.0f ? 0.0f : 1.0f / pc) : 1.0f, mean = pg * r, zl = cz * lse - pf;
        float d[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float w = a.renorm ? r * (g[i] - sel[i] * mean) : g[i] - mean;
            d[i] = keep ? x[i] * (f[i] + zl + w) : 0.0f;
        }
        const int64_t at = m;
        m += step;
        if (m0 + step < a.M) load();
        if (at < a.M) {
            T* out = (T*)a.dlogits + at * E;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (l * NE + i < E) out[l * NE + i] = f32_elem<DT>(d[i]);
        }
    }
}

template <int DT>
void route_grad(const MoeRouteGradArgs& a, hipStream_t s) {
    const int64_t n = (a.M + 15) / 16;
    const unsigned blocks = (unsigned)(n < 2048 ? n : 2048);
    if (a.E <= 16) route_grad_kernel<DT, 1><<<blocks, 256, 0, s>>>(a);
    else if (a.E <= 64) route_grad_kernel<DT, 4><<<blocks, 256, 0, s>>>(a);
    else if (a.E <= 128) route_grad_kernel<DT, 8><<<blocks, 256, 0, s>>>(a);
    else if (a.E <= 256) route_grad_kernel<DT, 16><<<blocks, 256, 0, s>>>(a);
    else route_grad_kernel<DT, 32><<<blocks, 256, 0, s>>>(a);
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
