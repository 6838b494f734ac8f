// Expert router (top-k of a softmax) and the expert layer of a few tokens.
//
//   route:  ids[m] = the k experts of largest logit (ties to the lower index),
//           w[m, s] = softmax(logits[m])[ids[m, s]], or renormalised over the k.
//   layer:  Y[m] = sum_s w[m, s] (act(X[m] Wg[e]) * (X[m] Wu[e])) Wd[e],  e = ids[m, s].
//
// The layer is two kernels.  The first routes (each workgroup the few tokens
// by itself: no kernel, no round trip through memory before the weights
// start to stream), takes the j-th expert in use and computes
// h = w act(gate) * up for every token that chose it, in fp32 to the
// workspace.  The second multiplies h by the down weights.
//
// Both are one read of the weights in use.  One token, 8 of 64 experts, 4096 x
// 2048 (bf16): 54 + 28 us for 268 + 134 MB; 32 tokens: 404 + 201 us for 2.1 +
// 1.1 GB, 5.4 TB/s, which is what the memory gives.  Small layers are bound by
// the steps around the stream: 23 tokens, 16 experts of 1024 x 1000 (fp16): 17 +
// 16 us, of which the weights take 11 + 8, routing 2, the join of the experts 4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"
#include "row_select.hpp"
#include "stream_core.hpp"

namespace omm {

namespace {

constexpr int kMaxE = 512;    // experts (32 logits a lane); checked by the caller
constexpr int kMaxTop = 16;   // selections a token
constexpr int kMaxTok = 64;   // tokens of a layer call: one lane each

// ------------------------------------------------------------------ routing
// 16 lanes a token, four tokens a wave: lane l holds the logits of experts NE l ..
// + NE - 1, so the lowest expert of a value is the lowest lane's.  A selection is
// two reductions over 16 lanes (largest key, lowest index) for four tokens at
// once, where a wave a token took one over 64 lanes each (16384 tokens over 64
// experts, 8 selections: 9.4 us; the selections' arithmetic was the time).
template <int DT, int NE>
__device__ __forceinline__ void load_logits(const typename elem_of<DT>::type* row, int E, int l, float (&x)[NE]) {
    if (E == 16 * NE) {
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = elem_f32<DT>(row[l * NE + i]);
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = l * NE + i < E ? elem_f32<DT>(row[l * NE + i]) : -__builtin_inff();
    }
}
// Lane l < k returns selection l (all 64 lanes must call)
template <int NE>
__device__ __forceinline__ void route_token(const float (&x)[NE], int E, int k, int renorm, int l, int& id, float& w) {
    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = l * NE + i < E ? order_key(x[i]) : 0;
    uint32_t first = 0, top = 0;
    id = 0;
    for (int s = 0; s < k; ++s) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) mx = max(mx, key[i]);
        mx = row16_max(mx);
        uint32_t e = 0xffffffffu;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
            if (key[i] == mx) e = l * NE + i;
        e = ~row16_max(~e);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (e == (uint32_t)(l * NE + i)) key[i] = 0;
        if (s == 0) first = mx;
        if (l == s) {
            id = (int)e;
            top = mx;
        }
    }
    const float mxv = key_value(first);
    const bool none = mxv == -__builtin_inff();  // every expert masked: all weights 0
    const float p = l < k ? expf(key_value(top) - mxv) : 0.0f;
    float z = p;
    if (!renorm) {
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (l * NE + i < E) z += expf(x[i] - mxv);
    }
    z = row16_sum(z);
    w = none ? 0.0f : p / z;
}

struct RouteArgs {
    const void* logits;
    void* ids;
    float* weights;
    int64_t M;
    int E, k, renorm, ids64;
};

template <int DT, int NE>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    const int l = threadIdx.x & 15;
    const int64_t m = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const bool here = m < a.M;
    float x[NE], w;
    int id;
    load_logits<DT, NE>((const typename elem_of<DT>::type*)a.logits + (here ? m : a.M - 1) * a.E, a.E, l, x);
    route_token<NE>(x, a.E, a.k, a.renorm, l, id, w);
    if (!here || l >= a.k) return;
    if (a.ids64) ((int64_t*)a.ids)[m * a.k + l] = id;
    else ((int32_t*)a.ids)[m * a.k + l] = id;
    a.weights[m * a.k + l] = w;
}

template <int DT>
void route_launch(const RouteArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.M + 15) / 16));
    if (a.E <= 16) route_kernel<DT, 1><<<grid, 256, 0, s>>>(a);
    else if (a.E <= 64) route_kernel<DT, 4><<<grid, 256, 0, s>>>(a);
    else if (a.E <= 128) route_kernel<DT, 8><<<grid, 256, 0, s>>>(a);
    else if (a.E <= 256) route_kernel<DT, 16><<<grid, 256, 0, s>>>(a);
    else route_kernel<DT, 32><<<grid, 256, 0, s>>>(a);
}

// ------------------------------------------------------------------ layer
// The (token, selection) pairs of one expert in use, as the first kernel
// leaves them to the second; ~pair where the weight is 0.  Such a pair adds
// nothing, whatever the expert's weights hold: 0 NaN would not be 0, and an
// excluded expert is selected where fewer than k others are left.
struct ExpertList {
    int32_t e, n, active, unused;
    int32_t pair[kMaxTok];
};
__device__ __forceinline__ int pair_of(int p) { return p ^ (p >> 31); }

struct LayerArgs {
    const void* X;         // (M, K)
    const void* logits;    // (M, E)
    const void* wg;        // trans 0: (E, K, F), 1: (E, F, K)
    const void* wu;
    const void* wd;        // trans 0: (E, F, K), 1: (E, K, F)
    void* Y;               // (M, K)
    int32_t* ids;          // workspace: (M, k) selections, -1 for those of weight 0 (element-wise form)
    ExpertList* lists;     // workspace: (min(E, M k)) (streamed form)
    float* hmax;           // workspace: (M k, ceil(F / hw)) largest |h| (fp16)
    float* h;              // workspace: (M k, F), weighted
    float* part;           // workspace: (ceil(K / 128), splits, M k, 128)
    uint32_t* done;        // workspace: finished workgroups of each 128 output columns
    int64_t K, F;
    int M, E, k, renorm, act, trans, logits_kind, splits;
    int hw;                // columns of a workgroup of the first kernel (16 or 64; streamed form)
};

__device__ __forceinline__ float activate(float g, int act) {
    if (act == 0) return g / (1.0f + expf(-g));                    // SiLU
    return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));     // GELU (erf)
}

// The tokens of the j-th expert in use (in ascending expert order)
struct ExpertRows {
    int32_t id[kMaxTok * kMaxTop];
    float w[kMaxTok * kMaxTop];
    uint32_t used[kMaxE / 32];
    int32_t tok[kMaxTok], slot[kMaxTok];
    int e, n, active;
};

// Routes the call's tokens, NW waves taking four each in turn
template <int DT, int NE, int NW>
__device__ __forceinline__ void route_tokens(const LayerArgs& a, ExpertRows& r, int lane, int wave) {
    const typename elem_of<DT>::type* logits = (const typename elem_of<DT>::type*)a.logits;
    const int l = lane & 15;
    for (int m0 = wave * 4; m0 < a.M; m0 += NW * 4) {
        const int m = m0 + (lane >> 4);
        float x[NE], w;
        int id;
        load_logits<DT, NE>(logits + min(m, a.M - 1) * a.E, a.E, l, x);
        route_token<NE>(x, a.E, a.k, a.renorm, l, id, w);
        if (m < a.M && l < a.k) {
            r.id[m * a.k + l] = id;
            r.w[m * a.k + l] = w;
        }
    }
}
template <int DT, int NW>
__device__ __forceinline__ void route_tokens(const LayerArgs& a, ExpertRows& r, int lane, int wave) {
    if (a.E <= 16) route_tokens<DT, 1, NW>(a, r, lane, wave);
    else if (a.E <= 64) route_tokens<DT, 4, NW>(a, r, lane, wave);
    else if (a.E <= 128) route_tokens<DT, 8, NW>(a, r, lane, wave);
    else route_tokens<DT, 32, NW>(a, r, lane, wave);
}
// (the logits may be of another type than the weights)
template <int NW>
__device__ __forceinline__ void route_all(const LayerArgs& a, ExpertRows& r, int lane, int wave) {
    if (a.logits_kind == 0) route_tokens<0, NW>(a, r, lane, wave);
    else if (a.logits_kind == 1) route_tokens<1, NW>(a, r, lane, wave);
    else route_tokens<2, NW>(a, r, lane, wave);
}

// From r.id (and a __syncthreads after it was written) to the rows of the j-th
// expert in use: r.e (-1: fewer experts in use), r.tok / r.slot / r.n.  All
// threads call it; it ends with a __syncthreads.
template <int NT>
__device__ __forceinline__ void expert_rows(ExpertRows& r, int M, int k, int j, int tid) {
    for (int i = tid; i < kMaxE / 32; i += NT) r.used[i] = 0;
    __syncthreads();
    for (int i = tid; i < M * k; i += NT) atomicOr(&r.used[r.id[i] >> 5], 1u << (r.id[i] & 31));
    __syncthreads();
    if (tid < 64) {
        const uint32_t word = tid < kMaxE / 32 ? r.used[tid] : 0;
        int before = __popc(word);  // inclusive prefix of the counts
#pragma unroll
        for (int d = 1; d < kMaxE / 32; d <<= 1) {
            const int o = __shfl_up(before, d, 64);
            if (tid >= d) before += o;
        }
        const int total = __shfl(before, kMaxE / 32 - 1, 64);
        before -= __popc(word);
        const bool here = tid < kMaxE / 32 && j >= before && j < before + __popc(word);
        int e = -1;
        if (here) {
            uint32_t v = word;
            for (int i = before; i < j; ++i) v &= v - 1;
            e = tid * 32 + __ffs(v) - 1;
        }
        e = wave_max(e);
        int slot = -1;
        if (e >= 0 && tid < M)
            for (int s = 0; s < k; ++s)
                if (r.id[tid * k + s] == e) slot = s;
        const uint64_t has = __ballot(slot >= 0);
        if (slot >= 0) {
            const int i = __popcll(has & ((1ull << tid) - 1));
            r.tok[i] = tid;
            r.slot[i] = slot;
        }
        if (tid == 0) {
            r.e = e;
            r.n = __popcll(has);
            r.active = total;
        }
    }
    __syncthreads();
}

// Element-wise forms: any sizes, alignments and types.  A workgroup computes
// 64 columns of one expert, lane = column, k split over its 4 waves.
template <int DT>
__global__ __launch_bounds__(256) void moe_up_any_kernel(LayerArgs a) {
    typedef typename elem_of<DT>::type E;
    __shared__ ExpertRows r;
    __shared__ float red[4][2][8][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    route_all<4>(a, r, lane, wave);
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = tid; i < a.M * a.k; i += 256) a.ids[i] = r.w[i] == 0.0f ? -1 : r.id[i];
    expert_rows<256>(r, a.M, a.k, (int)blockIdx.y, tid);
    if (r.e < 0) return;
    const int64_t f = (int64_t)blockIdx.x * 64 + lane;
    const int64_t sk = a.trans ? 1 : a.F, sf = a.trans ? a.K : 1;
    const int64_t base = (int64_t)r.e * a.K * a.F + (f < a.F ? f : 0) * sf;
    const E* wg = (const E*)a.wg + base;
    const E* wu = (const E*)a.wu + base;
    const int64_t kc = (a.K + 3) / 4, k0 = wave * kc, k1 = k0 + kc < a.K ? k0 + kc : a.K;
    for (int t0 = 0; t0 < r.n; t0 += 8) {
        float g[8] = {}, u[8] = {};
        const E* x[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) x[t] = (const E*)a.X + (int64_t)r.tok[min(t0 + t, r.n - 1)] * a.K;
        for (int64_t k = k0; k < k1; ++k) {
            const float vg = elem_f32<DT>(wg[k * sk]), vu = elem_f32<DT>(wu[k * sk]);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float xv = elem_f32<DT>(x[t][k]);
                g[t] = fmaf(xv, vg, g[t]);
                u[t] = fmaf(xv, vu, u[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            red[wave][0][t][lane] = g[t];
            red[wave][1][t][lane] = u[t];
        }
        __syncthreads();
        for (int i = tid; i < 8 * 64; i += 256) {
            const int t = i >> 6, c = i & 63;
            const int64_t fc = (int64_t)blockIdx.x * 64 + c;
            if (t0 + t < r.n && fc < a.F) {
                const float gv = red[0][0][t][c] + red[1][0][t][c] + red[2][0][t][c] + red[3][0][t][c];
                const float uv = red[0][1][t][c] + red[1][1][t][c] + red[2][1][t][c] + red[3][1][t][c];
                const int p = r.tok[t0 + t] * a.k + r.slot[t0 + t];
                a.h[(int64_t)p * a.F + fc] = activate(gv, a.act) * uv * r.w[p];
            }
        }
        __syncthreads();
    }
}

// A workgroup computes 64 columns of one token: its experts one after another
template <int DT>
__global__ __launch_bounds__(256) void moe_down_any_kernel(LayerArgs a) {
    typedef typename elem_of<DT>::type E;
    __shared__ float red[4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 + lane, m = blockIdx.y;
    const int64_t sf = a.trans ? 1 : a.K, sn = a.trans ? a.F : 1;
    const int64_t fc = (a.F + 3) / 4, f0 = wave * fc, f1 = f0 + fc < a.F ? f0 + fc : a.F;
    float acc = 0.0f;
    for (int s = 0; s < (a.F ? a.k : 0); ++s) {  // (no hidden columns: no first kernel, no selections)
        const int64_t p = m * a.k + s;
        if (a.ids[p] < 0) continue;
        const E* wd = (const E*)a.wd + (int64_t)a.ids[p] * a.K * a.F + (n < a.K ? n : 0) * sn;
        const float* h = a.h + p * a.F;
        for (int64_t f = f0; f < f1; ++f) acc = fmaf(h[f], elem_f32<DT>(wd[f * sf]), acc);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && n < a.K)
        ((E*)a.Y)[m * a.K + n] = f32_elem<DT>(red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane]);
}

template <int DT>
void layer_any(const LayerArgs& a, hipStream_t s) {
    const int pairs = a.M * a.k, jmax = pairs < a.E ? pairs : a.E;
    const dim3 gu((unsigned)((a.F + 63) / 64), (unsigned)jmax);
    if (a.F) moe_up_any_kernel<DT><<<gu, 256, 0, s>>>(a);
    const dim3 gd((unsigned)((a.K + 63) / 64), (unsigned)a.M);
    moe_down_any_kernel<DT><<<gd, 256, 0, s>>>(a);
}

// ------------------------------------------------------------------ streamed forms
// h of one expert and 64 columns: 64 gate columns and the 64 up columns beside
// them are the wave's 8 fragments, so that act(gate) * up needs no other
// workgroup.  TRANS = 0: lanes 0-7 of 16 load gate, 8-15 up (fp32: fragments
// 0-3 and 4-7); TRANS = 1: fragments 0-3 are gate, 4-7 up.
template <int DT, int TRANS, int NG, int NWS>
__device__ __forceinline__ void up_rows(const LayerArgs& a, const ExpertRows& r, int t0, float* red, int tid) {
    typedef typename elem_of<DT>::type E;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15;
    const int q = (lane >> 4) * kQ<DT>, tr = x_row<TRANS>(lane), tq = x_off<DT, TRANS>(lane);
    const int F = (int)a.F, K = (int)a.K, c0 = blockIdx.x * 64;
    const int64_t eoff = (int64_t)__builtin_amdgcn_readfirstlane(r.e) * a.K * a.F;
    const E* wg = (const E*)a.wg + eoff;
    const E* wu = (const E*)a.wu + eoff;
    StreamW<DT, TRANS> w;
    if constexpr (TRANS) {
        w.base[0] = wg;
        w.base[1] = wu;
#pragma unroll
        for (int j = 0; j < 8; ++j) w.off[j] = (uint32_t)min(c0 + 16 * (j & 3) + tr, F - 1) * K + tq;
    } else {
        w.ld = F;
        if constexpr (DT == 2) {
            w.p[0] = wg + group_start<DT>(c0, 4 * i, F) + (int64_t)q * F;
            w.p[1] = wu + group_start<DT>(c0, 4 * i, F) + (int64_t)q * F;
        } else {
            w.p[0] = (i < 8 ? wg : wu) + group_start<DT>(c0, 8 * (i & 7), F) + (int64_t)q * F;
        }
    }
    StreamX<DT, TRANS, NG> x;  // rows past the last are the last one: their results are not used
#pragma unroll
    for (int g = 0; g < NG; ++g)
        x.p[g] = (const E*)a.X + (int64_t)r.tok[min(t0 + 16 * g + tr, r.n - 1)] * K + tq;
    f32x4_t acc[8][NG] = {};
    int s0, s1;
    wave_steps<DT, NWS>(K, TRANS, wave, s0, s1);
    stream_run<DT, TRANS, NG>(w, x, s0, s1, K, acc, (u32x4_t*)&red[red_index(wave, 0, 0, 0)], lane);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g) __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) *(f32x4_t*)&red[red_index(wave, j, lane, 0)] = acc[j][g];
        __syncthreads();
        for (int o = tid; o < 16 * 64; o += 64 * NWS) {
            const int c = o & 63, row = o >> 6, t = t0 + 16 * g + row;
            if (t >= r.n) continue;  // a wave has one row
            int j, l, rr, j2, l2, rr2;
            const int shift = c0 + (c & ~(kQ<DT> - 1)) - group_start<DT>(c0, c, F);
            red_pos<DT, TRANS>(c, shift, row, j, l, rr);
            red_pos<DT, TRANS>(c + 64, shift, row, j2, l2, rr2);
            float gv = 0.0f, uv = 0.0f;
#pragma unroll
            for (int v = 0; v < NWS; ++v) {
                gv += red[red_index(v, j, l, rr)];
                uv += red[red_index(v, j2, l2, rr2)];
            }
            const int p = r.tok[t] * a.k + r.slot[t];
            const float h = c0 + c < F ? activate(gv, a.act) * uv * r.w[p] : 0.0f;
            if (c0 + c < F) a.h[(int64_t)p * F + c0 + c] = h;
            if constexpr (DT == 1) {
                const uint32_t mx = wave_max_u32(__float_as_uint(fabsf(h)));
                if (c == 0) a.hmax[(int64_t)p * gridDim.x + blockIdx.x] = __uint_as_float(mx);
            }
        }
    }
}

// The same for 16 columns: one gate and one up fragment, U steps on their way at
// once.  For few experts in use with a small F, where 64 columns would make few
// workgroups, each with a long contraction.
template <int DT, int TRANS, int NG>
__device__ __forceinline__ void up_cols(const LayerArgs& a, const ExpertRows& r, int t0, float* red, int tid) {
    typedef typename elem_of<DT>::type E;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int F = (int)a.F, K = (int)a.K, c0 = blockIdx.x * 16;
    const int64_t eoff = (int64_t)__builtin_amdgcn_readfirstlane(r.e) * a.K * a.F;
    const E* wg = (const E*)a.wg + eoff;
    const E* wu = (const E*)a.wu + eoff;
    ColsWeights<DT, TRANS, 2> w;
    if constexpr (TRANS) {
        w.base[0] = wg;
        w.base[1] = wu;
        w.off[0] = w.off[1] = (uint32_t)min(c0 + tile_row(lane), F - 1) * K + tile_off<DT>(lane);
    } else {
        constexpr int LPR = ColsW<DT, 2>::LPR;  // the first half of a row's lanes loads gate
        const int piece = lane % LPR;
        w.ld = F;
        w.p = (piece < LPR / 2 ? wg : wu) + (int64_t)(lane / LPR) * F + group_start<DT>(c0, piece % (LPR / 2) * kQ<DT>, F);
    }
    StreamX<DT, 1, NG> x;  // rows past the last are the last one: their results are not used
#pragma unroll
    for (int g = 0; g < NG; ++g)
        x.p[g] = (const E*)a.X + (int64_t)r.tok[min(t0 + 16 * g + tile_row(lane), r.n - 1)] * K + tile_off<DT>(lane);
    f32x4_t acc[2][NG] = {};
    int s0, s1;
    wave_steps<DT, 8>(K, 1, wave, s0, s1);
    cols_run<DT, TRANS, NG, 2, NG == 1 ? 4 : 2>(w, x, s0, s1, K, acc, (u32x4_t*)&red[red_index(wave, 0, 0, 0)], lane,
                                                [] {});
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < NG; ++g) *(f32x4_t*)&red[red_index(wave, 2 * j + g, lane, 0)] = acc[j][g];
    __syncthreads();
    for (int o = tid; o < 16 * NG * 16; o += 512) {
        const int c = o & 15, row = o >> 4, t = t0 + row;  // 16 lanes a row
        const int pos = cols_pos<DT, TRANS>(c0, c, F);
        float gv = 0.0f, uv = 0.0f;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            const float* q = &red[red_index(v, row >> 4, (pos >> 2) * 16 + (row & 15), pos & 3)];
            gv += q[0];
            uv += q[2 * kFragPad];
        }
        const bool in = t < r.n && c0 + c < F;
        const int p = t < r.n ? r.tok[t] * a.k + r.slot[t] : 0;
        const float h = in ? activate(gv, a.act) * uv * r.w[p] : 0.0f;
        if (in) a.h[(int64_t)p * F + c0 + c] = h;
        if constexpr (DT == 1) {
            const uint32_t mx = row16_max(__float_as_uint(fabsf(h)));
            if (c == 0 && t < r.n) a.hmax[(int64_t)p * gridDim.x + blockIdx.x] = __uint_as_float(mx);
        }
    }
}

template <int DT, int TRANS, int NG, int NWS, int CW>
__global__ __launch_bounds__(64 * NWS, NWS == 4 ? 3 : 2) void moe_up_kernel(LayerArgs a) {
    __shared__ ExpertRows r;
    __shared__ __attribute__((aligned(16))) float red[NWS * 8 * kFragPad];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    route_all<NWS>(a, r, lane, wave);
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0)  // for the second kernel, as the list below
        for (int i = tid; i < (a.K + 127) / 128; i += 64 * NWS) a.done[i] = 0;
    expert_rows<64 * NWS>(r, a.M, a.k, (int)blockIdx.y, tid);
    if (blockIdx.x == 0 && tid < 64) {
        ExpertList& l = a.lists[blockIdx.y];
        if (tid < r.n) {
            const int p = r.tok[tid] * a.k + r.slot[tid];
            l.pair[tid] = r.w[p] == 0.0f ? ~p : p;
        }
        if (tid == 0) {
            l.e = r.e;
            l.n = r.n;
            l.active = r.active;
        }
    }
    if (r.e < 0) return;
    for (int t0 = 0; t0 < r.n; t0 += 16 * NG) {
        if (t0) __syncthreads();
        if constexpr (CW == 16)
            up_cols<DT, TRANS, NG>(a, r, t0, red, tid);
        else
            up_rows<DT, TRANS, NG, NWS>(a, r, t0, red, tid);
    }
}

// part of one expert and 128 output columns
template <int DT, int TRANS, int NG, int NWS>
__device__ __forceinline__ void down_rows(const LayerArgs& a, const ExpertList& r, int t0, float* red, int tid) {
    typedef typename elem_of<DT>::type E;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15;
    const int q = (lane >> 4) * kQ<DT>, tr = x_row<TRANS>(lane), tq = x_off<DT, TRANS>(lane);
    const int F = (int)a.F, N = (int)a.K, c0 = blockIdx.x * 128;
    const E* wd = (const E*)a.wd + (int64_t)__builtin_amdgcn_readfirstlane(r.e) * a.K * a.F;
    StreamW<DT, TRANS> w;
    if constexpr (TRANS) {
        w.base[0] = w.base[1] = wd;
#pragma unroll
        for (int j = 0; j < 8; ++j) w.off[j] = (uint32_t)min(c0 + 16 * j + tr, N - 1) * F + tq;
    } else {
        w.ld = N;
        if constexpr (DT == 2) {
            w.p[0] = wd + group_start<DT>(c0, 4 * i, N) + (int64_t)q * N;
            w.p[1] = wd + group_start<DT>(c0, 64 + 4 * i, N) + (int64_t)q * N;
        } else {
            w.p[0] = wd + group_start<DT>(c0, 8 * i, N) + (int64_t)q * N;
        }
    }
    int s0, s1;
    const int sp = blockIdx.z;
    wave_steps<DT, NWS>(F, TRANS, wave, s0, s1, a.splits, sp);
    StreamXf<DT, TRANS, NG> x;
    float undo[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        x.p[g] = a.h + (int64_t)pair_of(r.pair[min(t0 + 16 * g + tr, r.n - 1)]) * F + x.off(lane);
        undo[g] = 1.0f;
        if constexpr (DT == 1) {  // the row's largest value over this wave's range -> [2^13, 2^14)
            const int slabs = (F + a.hw - 1) / a.hw;
            const int p = pair_of(r.pair[min(t0 + 16 * g + i, r.n - 1)]);
            float mx = 0.0f;
            for (int b = s0 * 32 / a.hw; b < min(slabs, (s1 * 32 + a.hw - 1) / a.hw); ++b) mx = fmaxf(mx, a.hmax[(int64_t)p * slabs + b]);
            const int ex = split_exp(mx);
            x.scale[g] = ldexpf(1.0f, ex);
            undo[g] = ldexpf(1.0f, -ex);
        }
    }
    f32x4_t acc[8][NG] = {};
    stream_run<DT, TRANS, NG>(w, x, s0, s1, F, acc, (u32x4_t*)&red[red_index(wave, 0, 0, 0)], lane);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        if (g) __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (DT == 1) acc[j][g] *= undo[g];
            *(f32x4_t*)&red[red_index(wave, j, lane, 0)] = acc[j][g];
        }
        __syncthreads();
        for (int o = tid; o < 16 * 128; o += 64 * NWS) {
            const int c = o & 127, row = o >> 7, t = t0 + 16 * g + row;
            if (t >= r.n || c0 + c >= N) continue;
            int j, l, rr;
            red_pos<DT, TRANS>(c, c0 + (c & ~(kQ<DT> - 1)) - group_start<DT>(c0, c, N), row, j, l, rr);
            float v = 0.0f;
#pragma unroll
            for (int u = 0; u < NWS; ++u) v += red[red_index(u, j, l, rr)];
            const int p = r.pair[t];
            part_store<128>(a.part, ((int64_t)blockIdx.x * a.splits + sp) * (a.M * a.k) + pair_of(p), c, p < 0 ? 0.0f : v);
        }
    }
}

// (4 waves a workgroup, trans 1, 16-bit weights: three waves a SIMD would spill; 32
// tokens over 64 experts of 4096 x 2048, the whole layer: bf16 849 us with three, 828
// with two, fp16 860 and 803)
template <int DT, int TRANS, int NG, int NWS>
__global__ __launch_bounds__(64 * NWS, NWS == 4 && !(TRANS && DT < 2) ? 3 : 2) void moe_down_kernel(LayerArgs a) {
    __shared__ ExpertList r;
    __shared__ __attribute__((aligned(16))) float red[NWS * 8 * kFragPad];
    const int tid = threadIdx.x;
    if (tid < (int)(sizeof(ExpertList) / 4)) ((int32_t*)&r)[tid] = ((const int32_t*)&a.lists[blockIdx.y])[tid];
    __syncthreads();
    if (r.e < 0) return;
    for (int t0 = 0; t0 < r.n; t0 += 16 * NG) {
        if (t0) __syncthreads();
        down_rows<DT, TRANS, NG, NWS>(a, r, t0, red, tid);
    }
    // The last workgroup of these 128 columns sums the experts (the first kernel
    // zeroed the count).
    if (!part_last(&a.done[blockIdx.x], r.active * a.splits, tid)) return;
    const int N = (int)a.K, k = a.k;
    part_sums<64 * NWS, 128>(
        a.part, a.M, k * a.splits, tid,
        [&](int m, int p) {
            const int sp = p / k;
            return ((int64_t)blockIdx.x * a.splits + sp) * (a.M * k) + m * k + (p - sp * k);
        },
        [&](int m, int c, float v0, float v1) {
            typedef typename elem_of<DT>::type E;
            const int n = blockIdx.x * 128 + c;
            E* y = (E*)a.Y + (int64_t)m * N + n;
            if (n < N) y[0] = f32_elem<DT>(v0);
            if (n + 1 < N) y[1] = f32_elem<DT>(v1);
        });
}

// NG groups of 16 tokens pass an expert's weights at once; an expert with more
// tokens reads them again (from the caches).
template <int DT, int TRANS, int NG, int NWS>
void layer_streamed(const LayerArgs& a, int jmax, hipStream_t s) {
    const dim3 gu((unsigned)((a.F + a.hw - 1) / a.hw), (unsigned)jmax);
    const dim3 gd((unsigned)((a.K + 127) / 128), (unsigned)jmax, (unsigned)a.splits);
    if constexpr (NWS == 8) {
        if (a.hw == 16) moe_up_kernel<DT, TRANS, NG, 8, 16><<<gu, 512, 0, s>>>(a);
        else moe_up_kernel<DT, TRANS, NG, 8, 64><<<gu, 512, 0, s>>>(a);
    } else {
        moe_up_kernel<DT, TRANS, NG, NWS, 64><<<gu, 64 * NWS, 0, s>>>(a);
    }
    moe_down_kernel<DT, TRANS, NG, NWS><<<gd, 64 * NWS, 0, s>>>(a);
}

// Workgroups that share one expert's 128 output columns by splitting F: as many
// as fill the chip, each wave with two steps of 32 or more.
int down_splits(int64_t M, int64_t K, int64_t F, int64_t E, int64_t k) {
    const int64_t jmax = M * k < E ? M * k : E, groups = (K + 127) / 128 * jmax;
    int64_t s = (256 + groups - 1) / groups;
    if (s > F / 256) s = F / 256;
    if (s > 4) s = 4;
    return s < 1 ? 1 : (int)s;
}

template <int DT, int TRANS>
void layer_pick(const LayerArgs& a, hipStream_t s) {
    const int pairs = a.M * a.k, jmax = pairs < a.E ? pairs : a.E;
    // two groups only where an expert has more than 8 tokens on average
    if (a.M > 16 && pairs > 8 * a.E) {
        layer_streamed<DT, TRANS, 2, 8>(a, jmax, s);
    } else if ((a.F + 63) / 64 * jmax <= 512) {
        layer_streamed<DT, TRANS, 1, 8>(a, jmax, s);
    } else {
        layer_streamed<DT, TRANS, 1, 4>(a, jmax, s);
    }
}

// whole groups of 8 columns, and one expert's matrix within 32-bit byte offsets
bool streamable(const LayerArgs& a, int dt) {
    return a.K >= 8 && a.F >= 8 && a.K * a.F < (dt == 2 ? 1LL << 29 : 1LL << 30);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs& r, int dt, hipStream_t s) {
    RouteArgs a;
    a.logits = r.logits;
    a.ids = r.ids;
    a.weights = r.weights;
    a.M = r.M;
    a.E = (int)r.E;
    a.k = r.k;
    a.renorm = r.renormalize;
    a.ids64 = r.ids64;
    if (dt == 0) route_launch<0>(a, s);
    else if (dt == 1) route_launch<1>(a, s);
    else route_launch<2>(a, s);
    return hipGetLastError();
}

size_t moe_layer_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t k) {
    const size_t jmax = (size_t)(M * k < E ? M * k : E);
    return align256((size_t)M * k * 4) + align256((size_t)M * k * F * 4) +
           align256((size_t)M * k * ((K + 127) / 128) * 512 * down_splits(M, K, F, E, k)) + align256((size_t)(K + 127) / 128 * 4) + align256(jmax * sizeof(ExpertList)) +
           align256((size_t)M * k * ((F + 15) / 16) * 4);
}

hipError_t launch_moe_layer(const MoeLayerArgs& l, int dt, int logits_kind, void* ws, hipStream_t s) {
    LayerArgs a;
    a.X = l.X;
    a.logits = l.logits;
    a.wg = l.w_gate;
    a.wu = l.w_up;
    a.wd = l.w_down;
    a.Y = l.Y;
    a.K = l.K;
    a.F = l.F;
    a.M = (int)l.M;
    a.E = (int)l.E;
    a.k = l.k;
    a.renorm = l.renormalize;
    a.act = l.activation;
    a.trans = l.trans;
    a.logits_kind = logits_kind;
    char* w = (char*)ws;
    a.ids = (int32_t*)w;
    w += align256((size_t)l.M * l.k * 4);
    a.h = (float*)w;
    w += align256((size_t)l.M * l.k * l.F * 4);
    a.part = (float*)w;
    a.splits = down_splits(l.M, l.K, l.F, l.E, l.k);
    // 64 columns of the first kernel, or 16 where that makes few workgroups (trans
    // 0, whose pieces of 16 columns are 32 bytes: fewer still).  us a call, 64 / 16
    // columns: trans 1, 2 experts of 2778 x 192 (6 workgroups of 64) fp32 40 / 23,
    // 13 of 3840 x 192 (39) 39 / 28, 3 of 512 x 1920 (90) 14 / 18; trans 0, 8 of
    // 2176 x 205 (32) 29 / 26, 16 of 896 x 192 (48) 16 / 20.
    const int64_t wide = (l.F + 63) / 64 * (l.M * l.k < l.E ? l.M * l.k : l.E);
    a.hw = wide < (l.trans ? 64 : 40) ? 16 : 64;
    w += align256((size_t)l.M * l.k * ((l.K + 127) / 128) * 512 * a.splits);
    a.done = (uint32_t*)w;
    w += align256((size_t)(l.K + 127) / 128 * 4);
    a.lists = (ExpertList*)w;
    w += align256((size_t)(l.M * l.k < l.E ? l.M * l.k : l.E) * sizeof(ExpertList));
    a.hmax = (float*)w;
    if (streamable(a, dt)) {
        log_choice("moe_layer: streamed");
        switch (dt * 2 + a.trans) {
            case 0: layer_pick<0, 0>(a, s); break;
            case 1: layer_pick<0, 1>(a, s); break;
            case 2: layer_pick<1, 0>(a, s); break;
            case 3: layer_pick<1, 1>(a, s); break;
            case 4: layer_pick<2, 0>(a, s); break;
            default: layer_pick<2, 1>(a, s); break;
        }
        return hipGetLastError();
    }
    log_choice("moe_layer: element-wise");
    if (dt == 0) layer_any<0>(a, s);
    else if (dt == 1) layer_any<1>(a, s);
    else layer_any<2>(a, s);
    return hipGetLastError();
}

}  // namespace omm
