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

// ------------------------------------------------------------------ counts and losses
// A workgroup's share: probabilities and counts by expert, and (sum lse^2, tokens).
struct Parts {
    float* p;        // [block][E]
    int32_t* count;  // [block][E]
    float* z;        // [block]
    int32_t* n;      // [block]
};
__host__ __device__ inline Parts parts_of(void* ws, int blocks, int E) {
    float* p = (float*)ws;
    int32_t* c = (int32_t*)(p + (int64_t)blocks * E);
    float* z = (float*)(c + (int64_t)blocks * E);
    return {p, c, z, (int32_t*)(z + blocks)};
}

template <int DT, int NE>
__global__ __launch_bounds__(256) void balance_parts_kernel(MoeBalanceArgs a, void* ws) {
    __shared__ int32_t count[kMaxE];
    __shared__ float psum[4][kMaxE];
    __shared__ float zsum[16];
    __shared__ int32_t nsum[16];
    const int t = threadIdx.x, l = t & 15, E = (int)a.E;
    for (int e = t; e < E; e += 256) count[e] = 0;
    __syncthreads();
    float p[NE] = {}, z = 0.0f;
    int n = 0;
    for (int64_t m0 = (int64_t)blockIdx.x * 16; m0 < a.M; m0 += (int64_t)gridDim.x * 16) {
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
    const int wave = t >> 6;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        p[i] += __shfl_xor(p[i], 16, 64);
        p[i] += __shfl_xor(p[i], 32, 64);
        if ((t & 63) < 16 && l * NE + i < E) psum[wave][l * NE + i] = p[i];
    }
    if (l == 0) {
        zsum[t >> 4] = z;
        nsum[t >> 4] = n;
    }
    __syncthreads();
    const Parts out = parts_of(ws, (int)gridDim.x, E);
    for (int e = t; e < E; e += 256) {
        out.p[(int64_t)blockIdx.x * E + e] = (psum[0][e] + psum[1][e]) + (psum[2][e] + psum[3][e]);
        out.count[(int64_t)blockIdx.x * E + e] = count[e];
    }
    if (t == 0) {
        float zs = 0.0f;
        int ns = 0;
        for (int i = 0; i < 16; ++i) {
            zs += zsum[i];
            ns += nsum[i];
        }
        out.z[blockIdx.x] = zs;
        out.n[blockIdx.x] = ns;
    }
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The join, one workgroup: thread t takes expert t % W of the parts t / W, t / W + 1024 / W ..
__global__ __launch_bounds__(1024) void balance_join_kernel(MoeBalanceArgs a, const void* ws, int blocks, int W) {
    __shared__ double ps[1024];
    __shared__ int32_t cs[1024];
    __shared__ double red[16][3];
    __shared__ int32_t redn[16];
    const int t = threadIdx.x, E = (int)a.E, e = t % W;
    const Parts in = parts_of((void*)ws, blocks, E);
    double p = 0.0, z = 0.0;
    int32_t c = 0, n = 0;
    if (e < E)
        for (int b = t / W; b < blocks; b += 1024 / W) {
            p += in.p[(int64_t)b * E + e];
            c += in.count[(int64_t)b * E + e];
        }
    for (int b = t; b < blocks; b += 1024) {
        z += in.z[b];
        n += in.n[b];
    }
    ps[t] = p;
    cs[t] = c;
    __syncthreads();
    double dot = 0.0, total = 0.0;
    if (t < W && e < E) {
        for (int i = t + W; i < 1024; i += W) {
            p += ps[i];
            c += cs[i];
        }
        a.counts[e] = c;
        dot = p * c;
        total = c;
    }
    dot = wave_sum64(dot);
    total = wave_sum64(total);
    z = wave_sum64(z);
#pragma unroll
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d, 64);
    if ((t & 63) == 0) {
        red[t >> 6][0] = dot;
        red[t >> 6][1] = total;
        red[t >> 6][2] = z;
        redn[t >> 6] = n;
    }
    __syncthreads();
    if (t == 0) {
        for (int i = 1; i < 16; ++i) {
            dot += red[i][0];
            total += red[i][1];
            z += red[i][2];
            n += redn[i];
        }
        // no token counted: both losses 0; no selection: the balance loss
        a.losses[0] = n && total > 0.0 ? (float)(E * (dot / total) / n) : 0.0f;
        a.losses[1] = n ? (float)(z / n) : 0.0f;
        a.tokens[0] = n;
    }
}

// Workgroups of the first kernel: 16 tokens each at a time; the second reads all
// their parts, 8 bytes an expert, so more experts get fewer of them.
int balance_blocks(int64_t M, int64_t E) {
    const int64_t most = E <= 64 ? 512 : E <= 128 ? 256 : 64;
    const int64_t n = (M + 15) / 16;
    return (int)(n < most ? n : most);
}

template <int DT>
void balance_parts(const MoeBalanceArgs& a, void* ws, int blocks, hipStream_t s) {
    if (a.E <= 16) balance_parts_kernel<DT, 1><<<blocks, 256, 0, s>>>(a, ws);
    else if (a.E <= 64) balance_parts_kernel<DT, 4><<<blocks, 256, 0, s>>>(a, ws);
    else if (a.E <= 128) balance_parts_kernel<DT, 8><<<blocks, 256, 0, s>>>(a, ws);
    else if (a.E <= 256) balance_parts_kernel<DT, 16><<<blocks, 256, 0, s>>>(a, ws);
    else balance_parts_kernel<DT, 32><<<blocks, 256, 0, s>>>(a, ws);
}

// ------------------------------------------------------------------ gradient
template <int DT, int NE>
__global__ __launch_bounds__(256) void route_grad_kernel(MoeRouteGradArgs a) {
    typedef typename elem_of<DT>::type T;
    __shared__ int32_t wsum[4];
    const int t = threadIdx.x, l = t & 15, E = (int)a.E, k = a.k;
    float f[NE] = {}, cz = 0.0f;
    if (a.g_losses) {
        int c = 0;
        for (int e = t; e < E; e += 256) c += a.counts[e];
#pragma unroll
        for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d, 64);
        if ((t & 63) == 0) wsum[t >> 6] = c;
        __syncthreads();
        const int total = wsum[0] + wsum[1] + wsum[2] + wsum[3], n = a.tokens[0];
        const float cb = n > 0 && total > 0 ? a.g_losses[0] * (float)E / (float)n : 0.0f;
        cz = n > 0 ? a.g_losses[1] * 2.0f / (float)n : 0.0f;
        // f of the formula with its factor
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (l * NE + i < E) f[i] = total > 0 ? cb * ((float)a.counts[l * NE + i] / (float)total) : 0.0f;
    }
    for (int64_t m0 = (int64_t)blockIdx.x * 16; m0 < a.M; m0 += (int64_t)gridDim.x * 16) {
        const int64_t m = m0 + (t >> 4);
        const bool here = m < a.M, keep = here && (!a.mask || a.mask[m]);
        float x[NE], g[NE] = {}, sel[NE] = {};
        load_row<DT, NE>(a.logits, here ? m : a.M - 1, E, l, x);
        if (a.g_weights) {
            int id = -1;
            float gs = 0.0f;
            if (keep && l < k) {
                const int64_t i = index_of(a.ids, m * k + l, a.ids64);
                if (i >= 0 && i < E) {
                    id = (int)i;
                    gs = a.g_weights[m * k + l];
                }
            }
            for (int s = 0; s < k; ++s) {
                const int e = __shfl(id, s, 16);
                const float v = __shfl(gs, s, 16);
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    g[i] += e == l * NE + i ? v : 0.0f;
                    sel[i] += e == l * NE + i ? 1.0f : 0.0f;
                }
            }
        }
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
        if (!here) continue;
        T* out = (T*)a.dlogits + m * E;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float w = a.renorm ? r * (g[i] - sel[i] * mean) : g[i] - mean;
            const float d = keep ? x[i] * (f[i] + zl + w) : 0.0f;
            if (l * NE + i < E) out[l * NE + i] = f32_elem<DT>(d);
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

size_t moe_balance_workspace_bytes(int64_t M, int64_t E) { return (size_t)balance_blocks(M, E) * (size_t)(8 * E + 8); }

hipError_t launch_moe_balance(const MoeBalanceArgs& a, int dt, void* ws, hipStream_t s) {
    const int blocks = balance_blocks(a.M, a.E);  // 0 for no tokens
    if (blocks == 0) {}
    else if (dt == 0) balance_parts<0>(a, ws, blocks, s);
    else if (dt == 1) balance_parts<1>(a, ws, blocks, s);
    else balance_parts<2>(a, ws, blocks, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int W = 16;
    while (W < a.E) W *= 2;
    balance_join_kernel<<<1, 1024, 0, s>>>(a, ws, blocks, W);
    return hipGetLastError();
}

hipError_t launch_moe_route_grad(const MoeRouteGradArgs& a, int dt, hipStream_t s) {
    if (dt == 0) route_grad<0>(a, s);
    else if (dt == 1) route_grad<1>(a, s);
    else route_grad<2>(a, s);
    return hipGetLastError();
}

}  // namespace omm
