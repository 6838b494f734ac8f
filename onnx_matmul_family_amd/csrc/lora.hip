// A shared projection with low-rank adapters chosen per row:
//   Y[m] = X[m] W (+ bias) + scale[g] (X[m] A[g]) B[g],   g = idx[m]
// (a row whose g is outside [0, G) has no adapter).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"
#include "row_select.hpp"

namespace omm {

namespace {

struct LoraK {
    const void* X;
    const void* A;
    const void* B;
    const void* idx;
    const float* scale;  // (G) or nullptr
    const void* bias;    // (N) or nullptr
    float* T;            // workspace: (M, R), scaled
    void* D;             // workspace: (M, N)
    int64_t M, K, N, G;
    int R, trans, idx64;
};

__device__ __forceinline__ int64_t row_adapter(const LoraK& a, int64_t m) {
    const int64_t g = a.idx64 ? ((const int64_t*)a.idx)[m] : (int64_t)((const int32_t*)a.idx)[m];
    return g >= 0 && g < a.G ? g : -1;
}

// T[m, r] = scale[g] sum_k X[m, k] A[g, k, r]: a workgroup a row, a wave an r
template <int DT>
__global__ __launch_bounds__(256) void lora_shrink_any_kernel(LoraK a) {
    typedef typename elem_of<DT>::type E;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = blockIdx.x, g = row_adapter(a, m);
    if (g < 0) return;
    const E* x = (const E*)a.X + m * a.K;
    const int64_t sk = a.trans ? 1 : a.R, sr = a.trans ? a.K : 1;
    for (int r = wave; r < a.R; r += 4) {
        const E* w = (const E*)a.A + g * a.K * a.R + r * sr;
        float acc = 0.0f;
        for (int64_t k = lane; k < a.K; k += 64) acc = fmaf(elem_f32<DT>(x[k]), elem_f32<DT>(w[k * sk]), acc);
        acc = wave_sum(acc);
        if (lane == 0) a.T[m * a.R + r] = a.scale ? acc * a.scale[g] : acc;
    }
}

// D[m, n] = bias[n] + sum_r T[m, r] B[g, r, n]
template <int DT>
__global__ __launch_bounds__(256) void lora_delta_any_kernel(LoraK a, int64_t nblk) {
    typedef typename elem_of<DT>::type E;
    const int64_t m = blockIdx.x / nblk, n = (blockIdx.x - m * nblk) * 256 + threadIdx.x;
    if (n >= a.N) return;
    const int64_t g = row_adapter(a, m);
    float acc = a.bias ? elem_f32<DT>(((const E*)a.bias)[n]) : 0.0f;
    if (g >= 0) {
        const int64_t sr = a.trans ? 1 : a.N, sn = a.trans ? a.R : 1;
        const E* b = (const E*)a.B + g * a.R * a.N + n * sn;
        const float* t = a.T + m * a.R;
        for (int r = 0; r < a.R; ++r) acc = fmaf(t[r], elem_f32<DT>(b[r * sr]), acc);
    }
    ((E*)a.D)[m * a.N + n] = f32_elem<DT>(acc);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R, int dt) {
    (void)K;
    return align256((size_t)M * R * 4) + align256((size_t)M * N * (dt == 2 ? 4 : 2));
}

hipError_t launch_lora(const LoraArgs& l, int dt, void* ws, hipStream_t s) {
    LoraK a;
    a.X = l.X;
    a.A = l.A;
    a.B = l.B;
    a.idx = l.idx;
    a.scale = l.scale;
    a.bias = l.bias;
    a.T = (float*)ws;
    a.D = (char*)ws + align256((size_t)l.M * l.R * 4);
    a.M = l.M;
    a.K = l.K;
    a.N = l.N;
    a.G = l.G;
    a.R = (int)l.R;
    a.trans = l.trans;
    a.idx64 = l.idx64;
    const int64_t nblk = (l.N + 255) / 256;
    const dim3 gs((unsigned)l.M), gd((unsigned)(l.M * nblk));
    if (dt == 0) {
        lora_shrink_any_kernel<0><<<gs, 256, 0, s>>>(a);
        lora_delta_any_kernel<0><<<gd, 256, 0, s>>>(a, nblk);
    } else if (dt == 1) {
        lora_shrink_any_kernel<1><<<gs, 256, 0, s>>>(a);
        lora_delta_any_kernel<1><<<gd, 256, 0, s>>>(a, nblk);
    } else {
        lora_shrink_any_kernel<2><<<gs, 256, 0, s>>>(a);
        lora_delta_any_kernel<2><<<gd, 256, 0, s>>>(a, nblk);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    DenseArgs d = {};
    d.A = l.X;
    d.B = l.W;
    d.Y = l.Y;
    d.C = a.D;
    d.M = l.M;
    d.N = l.N;
    d.K = l.K;
    d.lda = l.K;
    d.ldb = l.trans ? l.K : l.N;
    d.ldy = l.N;
    d.nb0 = d.nb1 = 1;
    d.c_sm = l.N;
    d.c_sn = 1;
    d.alpha = 1.0f;
    d.beta = 1.0f;
    d.a_kmajor = 1;
    d.b_kmajor = l.trans;
    return dt == 2 ? launch_dense_f32(d, s) : launch_dense16(d, dt, s);
}

}  // namespace omm
