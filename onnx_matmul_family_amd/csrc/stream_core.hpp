// Products of a few rows with a streamed weight matrix (bf16 / fp16): the
// weights pass from memory to the matrix unit once, with no LDS staging.
//
// A wave computes 8 fragments of 16 weight columns against groups of 16 rows,
// over a range of the contraction axis in steps of 32, with
// v_mfma_f32_16x16x32: the weights are the instruction's first operand (lane
// l: column l % 16 of the fragment, contraction 8 (l / 16) .. + 7), the rows
// its second, so lane l's results are row l % 16, columns 4 (l / 16) + r.
//
//   TRANS = 1: weights (columns, contraction), contraction contiguous.  A
//     fragment's operand is one 16-byte load a lane.
//   TRANS = 0: weights (contraction, columns), columns contiguous.  A lane
//     loads 16 bytes (8 columns) of each of 8 contraction rows: an 8 x 8 block
//     whose j-th columns, paired over the rows with v_perm (half an
//     instruction an element), are its operand of fragment j.  "Column l % 16"
//     of fragment j is then column 8 (l % 16) + j.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace omm {

template <int DT>
__device__ __forceinline__ f32x4_t mfma16x16x32(u32x4_t a, u32x4_t b, f32x4_t c) {
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// One lane's weights.  TRANS = 1: off[j], elements from base[j / 4] to the
// lane's column of fragment j; TRANS = 0: p, the lane's 8 columns, and ld, the
// row stride.  Both include the lane's contraction offset 8 (l / 16).  Bases,
// ld and kb are uniform over the wave (scalar registers).
template <int TRANS>
struct StreamW {
    const uint16_t* base[2];
    uint32_t off[8];
    __device__ __forceinline__ void load(u32x4_t (&w)[8], int kb) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = *(const u32x4_t*)(base[j >> 2] + kb + off[j]);
    }
};
template <>
struct StreamW<0> {
    const uint16_t* p;
    int64_t ld;
    __device__ __forceinline__ void load(u32x4_t (&w)[8], int kb) const {
        const uint16_t* q = p + (int64_t)kb * ld;
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = *(const u32x4_t*)(q + t * ld);
    }
};

template <int TRANS>
__device__ __forceinline__ u32x4_t stream_frag(const u32x4_t (&w)[8], int j) {
    if constexpr (TRANS) {
        return w[j];
    } else {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        u32x4_t f;
#pragma unroll
        for (int t = 0; t < 4; ++t) f[t] = __builtin_amdgcn_perm(w[2 * t + 1][j >> 1], w[2 * t][j >> 1], sel);
        return f;
    }
}

// The rows as stored: 16-bit values in the operand layout
template <int NG>
struct StreamX16 {
    static constexpr int RAW = 1, PARTS = 1;
    const uint16_t* p[NG];  // the lane's row of each group, offset by 8 (l / 16)
    __device__ __forceinline__ void load(u32x4_t (&r)[NG][1], int kb) const {
#pragma unroll
        for (int g = 0; g < NG; ++g) r[g][0] = *(const u32x4_t*)(p[g] + kb);
    }
    __device__ __forceinline__ void operand(const u32x4_t (&r)[1], int, u32x4_t (&o)[1]) const { o[0] = r[0]; }
};

// fp32 rows as the sum of two 16-bit halves (16 bits of the significand for
// bf16, 22 for fp16): two products instead of one, which the streamed weights
// leave room for, and the rows are not rounded to T.  fp16 rows are scaled by
// a power of two per row (scale[g]; the caller divides it out) into its range.
template <int DT, int NG>
struct StreamX32 {
    static constexpr int RAW = 2, PARTS = 2;
    const float* p[NG];
    float scale[NG];
    __device__ __forceinline__ void load(u32x4_t (&r)[NG][2], int kb) const {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            r[g][0] = *(const u32x4_t*)(p[g] + kb);
            r[g][1] = *(const u32x4_t*)(p[g] + kb + 4);
        }
    }
    __device__ __forceinline__ void operand(const u32x4_t (&r)[2], int g, u32x4_t (&o)[2]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = __uint_as_float(r[i >> 1][(i & 1) * 2]), b = __uint_as_float(r[i >> 1][(i & 1) * 2 + 1]);
            if constexpr (DT == 1) {
                a *= scale[g];
                b *= scale[g];
            }
            const uint32_t hi = pack2<DT>(a, b);
            const float ah = from_bits<DT>((uint16_t)hi), bh = from_bits<DT>((uint16_t)(hi >> 16));
            o[0][i] = hi;
            // an infinity is its own first half
            o[1][i] = pack2<DT>(a == ah ? 0.0f : a - ah, b == bh ? 0.0f : b - bh);
        }
    }
};

template <int DT, int TRANS, int NG, typename X>
__device__ __forceinline__ void stream_step(const u32x4_t (&w)[8], const u32x4_t (&r)[NG][X::RAW], const X& x,
                                            f32x4_t (&acc)[8][NG]) {
    u32x4_t o[NG][X::PARTS];
#pragma unroll
    for (int g = 0; g < NG; ++g) x.operand(r[g], g, o[g]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const u32x4_t f = stream_frag<TRANS>(w, j);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < X::PARTS; ++h) acc[j][g] = mfma16x16x32<DT>(f, o[g][h], acc[j][g]);
    }
}

// acc += steps [s0, s1) of 32 of a contraction of length kn (a multiple of 8;
// the last step may be partial: lanes past kn take zeros).  q8 = 8 (l / 16).
// Two register sets: the loads of a step are in flight while the one before
// it multiplies.
template <int DT, int TRANS, int NG, typename X>
__device__ __forceinline__ void stream_run(const StreamW<TRANS>& w, const X& x, int s0, int s1, int kn, int q8,
                                           f32x4_t (&acc)[8][NG]) {
    const int full = min(s1, kn >> 5);
    u32x4_t wa[8], wb[8], xa[NG][X::RAW], xb[NG][X::RAW];
    int s = s0;
    if (s < full) {
        w.load(wa, s * 32);
        x.load(xa, s * 32);
    }
    for (; s + 2 <= full; s += 2) {
        w.load(wb, s * 32 + 32);
        x.load(xb, s * 32 + 32);
        stream_step<DT, TRANS, NG>(wa, xa, x, acc);
        if (s + 2 < full) {
            w.load(wa, s * 32 + 64);
            x.load(xa, s * 32 + 64);
        }
        stream_step<DT, TRANS, NG>(wb, xb, x, acc);
    }
    if (s < full) {
        stream_step<DT, TRANS, NG>(wa, xa, x, acc);
        ++s;
    }
    if (s < s1 && s * 32 < kn) {  // partial last step
        const u32x4_t z = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) wa[j] = z;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < X::RAW; ++h) xa[g][h] = z;
        if (s * 32 + q8 < kn) {
            w.load(wa, s * 32);
            x.load(xa, s * 32);
        }
        stream_step<DT, TRANS, NG>(wa, xa, x, acc);
    }
}

// LDS image of a wave's 8 fragments of one group, for the sum over the waves
// that split the contraction: f32x4 at [wave][fragment][lane], one f32x4 of
// padding a fragment (reads that walk the fragments then change banks).
constexpr int kFragPad = 64 * 4 + 4;
__device__ __forceinline__ int red_index(int wave, int j, int lane, int r) {
    return (wave * 8 + j) * kFragPad + lane * 4 + r;
}
// position of (column c of the wave's 128, row of the group) in that image
template <int TRANS>
__device__ __forceinline__ void red_pos(int c, int row, int& j, int& lane, int& r) {
    const int i = TRANS ? c & 15 : c >> 3;
    j = TRANS ? c >> 4 : c & 7;
    lane = (i >> 2) * 16 + row;
    r = i & 3;
}

}  // namespace omm
