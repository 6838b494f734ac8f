// Argument block of the lora_matmul kernels (lora.hip: up to 64 rows and the
// element-wise form; lora_rows.hip: more rows).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace omm {

struct LoraK {
    const void* X;
    const void* W;
    const void* A;
    const void* B;
    const void* idx;
    const float* scale;  // (G) or nullptr
    const void* bias;    // (N) or nullptr
    void* Y;
    int64_t M, K, N, G;
    int R, trans, idx64, splits, cw;  // cw: columns of a workgroup (streamed form)
    // workspace
    float* T;        // (M, R), scaled; rows in the order of perm (up to 64 rows, trans 0: 4 of them to add up)
    float* part;     // (ceil(N / cw), splits, M, cw)
    uint32_t* done;  // finished workgroups of each cw columns
    int32_t* perm;   // (M) rows in the order of their adapters, or nullptr: as they come
    // bf16, fp16 over sorted rows, instead of T: its parts (3, M, R up to a multiple of 8,
    // zeros there), and (fp16) what a row's parts are multiplied by, for each 64 r
    uint16_t* Tp;
    float* undo;
};

// the adapter of row m, -1: none
__device__ __forceinline__ int64_t row_adapter(const LoraK& a, int64_t m) {
    const int64_t g = a.idx64 ? ((const int64_t*)a.idx)[m] : (int64_t)((const int32_t*)a.idx)[m];
    return g >= 0 && g < a.G ? g : -1;
}

// The streamed form takes 64 rows a group: `a` becomes the arguments of group z.
// (T: kParts buffers of 64 rows a group)
__device__ __forceinline__ void row_group(LoraK& a, int z, int parts, int elem) {
    const int64_t m0 = (int64_t)z * 64, blocks = (a.N + a.cw - 1) / a.cw;
    a.X = (const char*)a.X + m0 * a.K * elem;
    a.Y = (char*)a.Y + m0 * a.N * elem;
    a.idx = (const char*)a.idx + m0 * (a.idx64 ? 8 : 4);
    a.T += m0 * parts * a.R;
    a.part += m0 * blocks * a.splits * a.cw;
    a.done += z * blocks;
    a.M = a.M - m0 < 64 ? a.M - m0 : 64;
}

// Y = X W + C, C (M, N) of T (may be Y)
hipError_t lora_add_dense(const LoraK& a, const void* C, int dt, hipStream_t s);

// T by elements, of any sizes
void lora_shrink_any(const LoraK& a, int dt, hipStream_t s);

// whether lora_tile_kernel takes these operands
bool lora_tiles_ok(const LoraK& a, int dt);
// whether the forms of lora_rows.hip take these sizes (of up to 2^20 rows)
bool lora_rows_ok(int64_t K, int64_t N, int64_t R, int64_t G);
size_t lora_rows_workspace_bytes(int64_t M, int64_t R);
hipError_t launch_lora_rows(LoraK a, int dt, void* ws, hipStream_t s);

}  // namespace omm
