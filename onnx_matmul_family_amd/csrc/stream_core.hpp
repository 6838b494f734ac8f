// Products of a few rows with a streamed weight matrix: the weights pass from
// memory to the matrix unit once, with no LDS staging.
//
// A wave computes NF (8, or fewer with TRANS = 1) fragments of 16 weight columns against groups of 16 rows,
// over a range of the contraction axis.  The weights are the instruction's
// first operand, the rows its second, so lane l's results are row l % 16,
// columns 4 (l / 16) + r of a fragment.
//
// bf16 / fp16, v_mfma_f32_16x16x32, steps of 32 (lane l: column l % 16,
// contraction 8 (l / 16) .. + 7):
//   TRANS = 1: weights (columns, contraction), contraction contiguous.  A
//     fragment's operand is one 16-byte load a lane (through row_tile below).
//   TRANS = 0: weights (contraction, columns), columns contiguous.  A lane
//     loads 16 bytes (8 columns) of each of 8 contraction rows: an 8 x 8 block
//     whose j-th columns, paired over the rows with v_perm (half an
//     instruction an element), are its operand of fragment j.  "Column l % 16"
//     of fragment j is then column 8 (l % 16) + j.
// fp32, v_mfma_f32_16x16x4, steps of 16 (an instruction takes one value of
// each lane, so a step is four of them; contraction 4 (l / 16) + t in the t-th):
//   TRANS = 1: as above, 4 values a load, the t-th for the t-th instruction.
//   TRANS = 0: a lane loads 4 columns of each of 4 contraction rows, twice (64
//     columns apart); fragment j takes the (j % 4)-th value, "column l % 16" is
//     column 64 (j / 4) + 4 (l % 16) + j % 4.
//
// Rows and columns need no alignment beyond their elements' (the loads are
// 16 bytes wide all the same), sizes no multiples: a TRANS = 0 lane whose
// columns pass the last one starts at the last whole group instead, and the
// tail of the contraction is loaded element by element.
//
// Loads of rows (the weights of TRANS = 1, and the rows X): in the operand's
// order 16 neighbouring lanes would read 16 different rows, and the caches look
// up a line for every lane (measured: 7 bytes a clock and CU, the rate of the
// memory itself).  So 4 neighbouring lanes read 64 bytes of one row, and the
// values take their operand places through LDS (1 KiB a fragment, of the wave's
// own, no barrier).  With TRANS = 0 only the rows X are loaded like that, which
// are few lines beside the weights': they are read in the operand's order (32
// tokens over 64 experts: up projection 407 us, through LDS 422).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "row_select.hpp"

namespace omm {

// 16 bytes at any multiple of the element size
typedef u32x4_t u32x4_u2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_u4 __attribute__((aligned(4)));
template <typename E>
__device__ __forceinline__ u32x4_t load16(const E* p) {
    if constexpr (sizeof(E) == 2)
        return *(const u32x4_u2*)p;
    else
        return *(const u32x4_u4*)p;
}
// the first n elements of those 16 bytes, zeros after them
template <typename E>
__device__ __forceinline__ u32x4_t load16_first(const E* p, int n) {
    u32x4_t v = {0, 0, 0, 0};
    if (n >= (int)(16 / sizeof(E))) return load16(p);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(E)); ++i) {
        if (i >= n) continue;
        if constexpr (sizeof(E) == 2)
            v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        else
            v[i] = __float_as_uint(p[i]);
    }
    return v;
}

template <int DT> constexpr int kStep = DT == 2 ? 16 : 32;  // contraction of a step
template <int DT> constexpr int kQ = DT == 2 ? 4 : 8;       // of one lane

template <int DT>
__device__ __forceinline__ f32x4_t mfma16x16x32(u32x4_t a, u32x4_t b, f32x4_t c) {
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Row and 16-byte piece of its 64 bytes that a lane loads of a tile of 16 rows;
// the pieces are permuted so that the read back meets every LDS bank once.
__device__ __forceinline__ int tile_row(int lane) { return lane >> 2; }
__device__ __forceinline__ int tile_piece(int lane) { return (lane & 3) ^ (lane >> 4); }
// where the tile's (row, piece) is among the lanes
__device__ __forceinline__ int tile_slot(int row, int piece) { return 4 * row + (piece ^ (row >> 2)); }
// contraction offset of the piece
template <int DT>
__device__ __forceinline__ int tile_off(int lane) { return tile_piece(lane) * kQ<DT>; }

// v[j] (tile j as loaded) -> lane l's 16 bytes of row l % 16, piece l / 16
template <int N>
__device__ __forceinline__ void row_tile(u32x4_t (&v)[N], u32x4_t* scratch, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j) scratch[j * 64 + lane] = v[j];
    __builtin_amdgcn_wave_barrier();
    const int slot = tile_slot(lane & 15, lane >> 4);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = scratch[j * 64 + slot];
    __builtin_amdgcn_wave_barrier();
}

// One lane's weights.  TRANS = 1: off[j], elements from base[2 j / NF] to the
// tile row's column of fragment j, plus the contraction offset tile_off;
// TRANS = 0: p, the lane's columns (fp32: p[1] of the upper 64), plus rows
// kQ (l / 16), and ld, the row stride.  Bases, ld and kb are uniform over the
// wave (scalar registers).  tail: of a contraction that ends at kn.
template <int DT, int TRANS, int NF = 8>
struct StreamW {
    typedef typename elem_of<DT>::type E;
    const E* base[2];
    uint32_t off[NF];
    __device__ __forceinline__ void load(u32x4_t (&w)[NF], int kb) const {
#pragma unroll
        for (int j = 0; j < NF; ++j) w[j] = load16(base[2 * j / NF] + kb + off[j]);
    }
    __device__ __forceinline__ void tail(u32x4_t (&w)[NF], int kb, int kn, int lane) const {
        const int n = max(0, min(kQ<DT>, kn - kb - tile_off<DT>(lane)));
#pragma unroll
        for (int j = 0; j < NF; ++j) w[j] = load16_first(base[2 * j / NF] + kb + off[j], n);
    }
};
template <int DT>
struct StreamW<DT, 0, 8> {
    typedef typename elem_of<DT>::type E;
    const E* p[DT == 2 ? 2 : 1];
    int64_t ld;
    __device__ __forceinline__ const E* at(int kb, int t) const {
        if constexpr (DT == 2)
            return p[t >> 2] + (int64_t)kb * ld + (t & 3) * ld;
        else
            return p[0] + (int64_t)kb * ld + t * ld;
    }
    __device__ __forceinline__ void load(u32x4_t (&w)[8], int kb) const {
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = load16(at(kb, t));
    }
    __device__ __forceinline__ void tail(u32x4_t (&w)[8], int kb, int kn, int lane) const {
        const int n = kn - kb - (lane >> 4) * kQ<DT>;
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = (t & (kQ<DT> - 1)) < n ? load16(at(kb, t)) : u32x4_t{0, 0, 0, 0};
    }
};

// bf16 / fp16: a lane's operand of fragment j
template <int TRANS, int NF>
__device__ __forceinline__ u32x4_t stream_frag(const u32x4_t (&w)[NF], int j) {
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

// row of 16 and contraction offset (16-byte pieces of 4 bytes: 4 values; of T:
// kQ) that a lane loads of the rows X
template <int TRANS>
__device__ __forceinline__ int x_row(int lane) { return TRANS ? tile_row(lane) : lane & 15; }
template <int DT, int TRANS>
__device__ __forceinline__ int x_off(int lane) { return TRANS ? tile_off<DT>(lane) : (lane >> 4) * kQ<DT>; }

// The rows as stored
template <int DT, int TRANS, int NG>
struct StreamX {
    static constexpr int RAW = 1, PARTS = 1;
    typedef typename elem_of<DT>::type E;
    const E* p[NG];  // row x_row of each group, plus off
    __device__ __forceinline__ static int off(int lane) { return x_off<DT, TRANS>(lane); }
    __device__ __forceinline__ void load(u32x4_t (&r)[NG][1], int kb) const {
#pragma unroll
        for (int g = 0; g < NG; ++g) r[g][0] = load16(p[g] + kb);
    }
    __device__ __forceinline__ void tail(u32x4_t (&r)[NG][1], int kb, int kn, int lane) const {
        const int n = max(0, min(kQ<DT>, kn - kb - off(lane)));
#pragma unroll
        for (int g = 0; g < NG; ++g) r[g][0] = load16_first(p[g] + kb, n);
    }
    __device__ __forceinline__ void operands(const u32x4_t (&r)[NG][1], u32x4_t (&o)[NG][1], u32x4_t* scratch,
                                             int lane) const {
        u32x4_t v[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) v[g] = r[g][0];
        if constexpr (TRANS) row_tile<NG>(v, scratch, lane);
#pragma unroll
        for (int g = 0; g < NG; ++g) o[g][0] = v[g];
    }
};

// Eight fp32 values as three parts of T each, which add up to them: 3 x 8 bits of
// the significand (bf16) or 3 x 11 (fp16, whose caller has scaled the row's
// largest value into its range; what is lost is 2^-37 of that one).  Two parts
// are not enough: 16 bits of a bf16 row made 600 of 131072 outputs of an expert
// layer (32 tokens, 4096 x 2048) miss the nearest bf16.  bf16 parts are
// cut off, not rounded: a value near the largest float stays finite.  An infinity
// is its own first part.
constexpr int kParts32 = 3;
template <int DT> constexpr float kLeastPart = DT == 1 ? 0x1p-24f : 0x1p-133f;
// |v| or, if that is less or NaN (inf - inf), the least part, unless z is 0; z's sign
template <int DT>
__device__ __forceinline__ float at_least(float v, float z) {
    return copysignf(fmaxf(fabsf(v), fminf(fabsf(z), kLeastPart<DT>)), z);
}
// what is less than the least part is raised to it (fp16, whose rows are scaled)
template <int DT>
__device__ __forceinline__ float split_raise(float v) {
    if (DT == 1 && fabsf(v) < kLeastPart<DT> && v != 0.0f) return copysignf(kLeastPart<DT>, v);
    return v;
}
// the next part of two values (a in the low half), which keep what is left of them
template <int DT>
__device__ __forceinline__ uint32_t split_pair(float& a, float& b) {
    uint32_t p;
    float ah, bh;
    if constexpr (DT == 1) {
        p = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
        ah = from_bits<DT>((uint16_t)p);
        bh = from_bits<DT>((uint16_t)(p >> 16));
    } else {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        p = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        ah = __uint_as_float(ua & 0xffff0000u);
        bh = __uint_as_float(ub & 0xffff0000u);
    }
    a = at_least<DT>(a - ah, ah);
    b = at_least<DT>(b - bh, bh);
    return p;
}
template <int DT>
__device__ __forceinline__ void split_parts(const u32x4_t (&r)[2], float scale, u32x4_t (&p)[kParts32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = __uint_as_float(r[i >> 1][(i & 1) * 2]), b = __uint_as_float(r[i >> 1][(i & 1) * 2 + 1]);
        if constexpr (DT == 1) {
            a = split_raise<DT>(a * scale);
            b = split_raise<DT>(b * scale);
        }
#pragma unroll
        for (int h = 0; h < kParts32; ++h) p[h][i] = split_pair<DT>(a, b);
    }
}
// the power of two that takes a row's largest value to [2^13, 2^14) (fp16)
__device__ __forceinline__ int split_exp(float mx) {
    return mx > 0.0f && mx < __builtin_inff() ? max(-100, min(100, 13 - ilogbf(mx))) : 0;
}

// fp32 rows against bf16 / fp16 weights, as the sum of three 16-bit parts: three
// products instead of one, which the streamed weights leave room for, and the
// rows are not rounded.  fp16 rows are scaled by a power of two per row
// (scale[g], of row l % 16; the caller divides it out).  Two loads a step:
// TRANS = 1 two tiles of 16 values of the contraction each, else 8 values.
template <int DT, int TRANS, int NG>
struct StreamX32 {
    static constexpr int RAW = 2, PARTS = kParts32, NEXT = TRANS ? 16 : 4;
    const float* p[NG];  // row x_row, plus off
    float scale[NG];
    __device__ __forceinline__ static int off(int lane) { return TRANS ? 4 * tile_piece(lane) : (lane >> 4) * 8; }
    __device__ __forceinline__ void load(u32x4_t (&r)[NG][2], int kb) const {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            r[g][0] = load16(p[g] + kb);
            r[g][1] = load16(p[g] + kb + NEXT);
        }
    }
    __device__ __forceinline__ void tail(u32x4_t (&r)[NG][2], int kb, int kn, int lane) const {
        const int n = kn - kb - off(lane);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            r[g][0] = load16_first(p[g] + kb, n);
            r[g][1] = load16_first(p[g] + kb + NEXT, n - NEXT);
        }
    }
    __device__ __forceinline__ void operands(const u32x4_t (&r)[NG][2], u32x4_t (&o)[NG][PARTS], u32x4_t* scratch,
                                             int lane) const {
        if constexpr (TRANS) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                scratch[2 * g * 64 + lane] = r[g][0];
                scratch[(2 * g + 1) * 64 + lane] = r[g][1];
            }
            __builtin_amdgcn_wave_barrier();
        }
        // contraction 8 (l / 16) .. + 7: pieces 2 (l / 16) and the next of the 8
        const int i = lane & 15, q = lane >> 4, h = (q >> 1) * 64;
        const int s0 = h + tile_slot(i, 2 * (q & 1)), s1 = h + tile_slot(i, 2 * (q & 1) + 1);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if constexpr (TRANS) {
                const u32x4_t v[2] = {scratch[2 * g * 64 + s0], scratch[2 * g * 64 + s1]};
                split_parts<DT>(v, scale[g], o[g]);
            } else {
                split_parts<DT>(r[g], scale[g], o[g]);
            }
        }
        if constexpr (TRANS) __builtin_amdgcn_wave_barrier();
    }
};
// The same from rows that are split already: p in the first part's rows, the next
// parts `plane` elements further on each.
template <int DT, int TRANS, int NG>
struct StreamXParts {
    static constexpr int RAW = kParts32, PARTS = kParts32;
    typedef typename elem_of<DT>::type E;
    const E* p[NG];  // row x_row, plus off
    int64_t plane;
    __device__ __forceinline__ static int off(int lane) { return x_off<DT, TRANS>(lane); }
    __device__ __forceinline__ void load(u32x4_t (&r)[NG][RAW], int kb) const {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < RAW; ++h) r[g][h] = load16(p[g] + h * plane + kb);
    }
    __device__ __forceinline__ void tail(u32x4_t (&r)[NG][RAW], int kb, int kn, int lane) const {
        const int n = max(0, min(kQ<DT>, kn - kb - off(lane)));
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int h = 0; h < RAW; ++h) r[g][h] = load16_first(p[g] + h * plane + kb, n);
    }
    __device__ __forceinline__ void operands(const u32x4_t (&r)[NG][RAW], u32x4_t (&o)[NG][PARTS], u32x4_t* scratch,
                                             int lane) const {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            u32x4_t v[PARTS];
#pragma unroll
            for (int h = 0; h < PARTS; ++h) v[h] = r[g][h];
            if constexpr (TRANS) row_tile<PARTS>(v, scratch, lane);
#pragma unroll
            for (int h = 0; h < PARTS; ++h) o[g][h] = v[h];
        }
    }
};
template <int DT, int TRANS, int NG>
using StreamXf = typename std::conditional<DT == 2, StreamX<2, TRANS, NG>, StreamX32<DT, TRANS, NG>>::type;

// (w is used up: its tiles are put in place)
template <int DT, int TRANS, int NG, int NF, typename X>
__device__ __forceinline__ void stream_step(u32x4_t (&w)[NF], const u32x4_t (&r)[NG][X::RAW], const X& x,
                                            f32x4_t (&acc)[NF][NG], u32x4_t* scratch, int lane) {
    u32x4_t o[NG][X::PARTS];
    x.operands(r, o, scratch, lane);
    if constexpr (TRANS) row_tile<NF>(w, scratch, lane);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        if constexpr (DT == 2) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t wv;
                    if constexpr (TRANS)
                        wv = w[j][t];
                    else
                        wv = w[(j >> 2) * 4 + t][j & 3];
                    acc[j][g] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(wv), __uint_as_float(o[g][0][t]),
                                                                     acc[j][g], 0, 0, 0);
                }
        } else {
            const u32x4_t f = stream_frag<TRANS, NF>(w, j);
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int h = 0; h < X::PARTS; ++h) acc[j][g] = mfma16x16x32<DT>(f, o[g][h], acc[j][g]);
        }
    }
}

// acc += steps [s0, s1) of kStep of a contraction of length kn (the last step
// may be partial: the lanes take zeros past kn).  scratch: LDS of this wave's
// own, 1 KiB each for the larger of NF (TRANS = 1) and NG X::RAW tiles.
// Two register sets: the loads of a step are in flight while the one before
// it multiplies.  `meanwhile` runs while the first weights are on their way (it
// may still set x).
template <int DT, int TRANS, int NG, typename X, int NF, typename F>
__device__ __forceinline__ void stream_run(const StreamW<DT, TRANS, NF>& w, const X& x, int s0, int s1, int kn,
                                           f32x4_t (&acc)[NF][NG], u32x4_t* scratch, int lane, F meanwhile) {
    constexpr int ST = kStep<DT>;
    const int full = min(s1, kn / ST);
    u32x4_t wa[NF], wb[NF], xa[NG][X::RAW], xb[NG][X::RAW];
    int s = s0;
    if (s < full) w.load(wa, s * ST);
    meanwhile();
    if (s < full) x.load(xa, s * ST);
    for (; s + 2 <= full; s += 2) {
        w.load(wb, s * ST + ST);
        x.load(xb, s * ST + ST);
        stream_step<DT, TRANS, NG, NF>(wa, xa, x, acc, scratch, lane);
        if (s + 2 < full) {
            w.load(wa, s * ST + 2 * ST);
            x.load(xa, s * ST + 2 * ST);
        }
        stream_step<DT, TRANS, NG, NF>(wb, xb, x, acc, scratch, lane);
    }
    if (s < full) {
        stream_step<DT, TRANS, NG, NF>(wa, xa, x, acc, scratch, lane);
        ++s;
    }
    if (s < s1 && s * ST < kn) {  // partial last step
        w.tail(wa, s * ST, kn, lane);
        x.tail(xa, s * ST, kn, lane);
        stream_step<DT, TRANS, NG, NF>(wa, xa, x, acc, scratch, lane);
    }
}

template <int DT, int TRANS, int NG, typename X, int NF>
__device__ __forceinline__ void stream_run(const StreamW<DT, TRANS, NF>& w, const X& x, int s0, int s1, int kn,
                                           f32x4_t (&acc)[NF][NG], u32x4_t* scratch, int lane) {
    stream_run<DT, TRANS, NG>(w, x, s0, s1, kn, acc, scratch, lane, [] {});
}

// first column of the lane group that holds column c0 + c (c in 0 .. span) of
// an axis of n columns: groups of kQ start at multiples, the last one at n - kQ
template <int DT>
__device__ __forceinline__ int group_start(int c0, int c, int n) {
    return min(c0 + (c & ~(kQ<DT> - 1)), n - kQ<DT>);
}

// contraction steps of one of a workgroup's NWS waves: even counts where a
// 128-byte line of a weight column holds two
template <int DT, int NWS>
__device__ __forceinline__ void wave_steps(int kn, int trans, int wave, int& s0, int& s1, int splits = 1,
                                           int split = 0) {
    const int steps = (kn + kStep<DT> - 1) / kStep<DT>, n = NWS * splits;
    int per = (steps + n - 1) / n;
    if (trans) per = (per + 1) & ~1;
    s0 = min(steps, (split * NWS + wave) * per);
    s1 = min(steps, s0 + per);
}

// LDS image of a wave's 8 fragments of one group, for the sum over the waves
// that split the contraction: f32x4 at [wave][fragment][lane], one f32x4 of
// padding a fragment (reads that walk the fragments then change banks).
constexpr int kFragPad = 64 * 4 + 4;
__device__ __forceinline__ int red_index(int wave, int j, int lane, int r) {
    return (wave * 8 + j) * kFragPad + lane * 4 + r;
}
// position of (column c of the wave's 128, row of the group) in that image;
// shift: how far before its multiple the column's group starts
template <int DT, int TRANS>
__device__ __forceinline__ void red_pos(int c, int shift, int row, int& j, int& lane, int& r) {
    int i;
    if constexpr (TRANS) {
        i = c & 15;
        j = c >> 4;
    } else if constexpr (DT == 2) {
        i = (c & 63) >> 2;
        j = (c >> 6) * 4 + min((c & 3) + shift, 3);
    } else {
        i = c >> 3;
        j = min((c & 7) + shift, 7);
    }
    lane = (i >> 2) * 16 + row;
    r = i & 3;
}

// ------------------------------------------------------------------ few columns
// 16 NF columns (NF 1, 2 or 4) against NG groups of 16 rows.  A step is few loads
// of the weights beside NG of the rows, so U steps are on their way at once in
// each of two register sets, and the rows take row_tile in either layout.
//   TRANS = 1: the weights too (StreamW).
//   TRANS = 0: a load takes 16-byte pieces of 32 / NF contraction rows (fp32:
//     16 / NF); in LDS they lie as in memory and are read by columns (16 bits:
//     the transposing read).
template <int DT, int NF>
struct ColsW {
    typedef typename elem_of<DT>::type E;
    static constexpr int LPR = NF * (DT == 2 ? 4 : 2), ROWS = 64 / LPR;  // lanes a row, rows a load
    const E* p;  // the lane's row and columns
    int64_t ld;
    __device__ __forceinline__ void load(u32x4_t (&w)[NF], int kb) const {
#pragma unroll
        for (int j = 0; j < NF; ++j) w[j] = load16(p + (int64_t)(kb + j * ROWS) * ld);
    }
    __device__ __forceinline__ void tail(u32x4_t (&w)[NF], int kb, int kn, int lane) const {
#pragma unroll
        for (int j = 0; j < NF; ++j)
            w[j] = kb + j * ROWS + lane / LPR < kn ? load16(p + (int64_t)(kb + j * ROWS) * ld) : u32x4_t{0, 0, 0, 0};
    }
    // tiles as loaded -> operands of the NF fragments
    __device__ __forceinline__ static void operands(u32x4_t (&w)[NF], u32x4_t* scratch, int lane) {
        constexpr int RB = LPR * 16;  // bytes a row
#pragma unroll
        for (int j = 0; j < NF; ++j) scratch[j * 64 + lane] = w[j];
        __builtin_amdgcn_wave_barrier();
        const int i = lane & 15, q = lane >> 4;
        const char* b = (const char*)scratch;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            if constexpr (DT == 2) {
#pragma unroll
                for (int t = 0; t < 4; ++t) w[j][t] = *(const uint32_t*)(b + (4 * q + t) * RB + j * 64 + 4 * i);
            } else {
                const char* f = b + (8 * q + (i >> 2)) * RB + j * 32 + 8 * (i & 3);
                const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OMM_LDS(i16x4_t, f));
                const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(OMM_LDS(i16x4_t, f + 4 * RB));
                const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
                w[j] = u32x4_t{l2.x, l2.y, h2.x, h2.y};
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
};

template <int DT, int TRANS, int NF>
using ColsWeights = typename std::conditional<TRANS != 0, StreamW<DT, 1, NF>, ColsW<DT, NF>>::type;

// weights of the columns from c0 on: TRANS = 1 (n, k), 0 (k, n)
template <int DT, int TRANS, int NF>
__device__ __forceinline__ void cols_start(ColsWeights<DT, TRANS, NF>& w, const typename elem_of<DT>::type* p, int c0,
                                           int n, int k, int lane) {
    if constexpr (TRANS) {
        w.base[0] = w.base[1] = p;
#pragma unroll
        for (int j = 0; j < NF; ++j) w.off[j] = (uint32_t)min(c0 + 16 * j + tile_row(lane), n - 1) * k + tile_off<DT>(lane);
    } else {
        constexpr int LPR = ColsW<DT, NF>::LPR;
        w.ld = n;
        w.p = p + (int64_t)(lane / LPR) * n + group_start<DT>(c0, (lane % LPR) * kQ<DT>, n);
    }
}
// column c's place among the workgroup's (a group of columns may start before its multiple)
template <int DT, int TRANS>
__device__ __forceinline__ int cols_pos(int c0, int c, int n) {
    if constexpr (TRANS) return c;
    const int g = c & ~(kQ<DT> - 1);
    return g + min((c - g) + c0 + g - group_start<DT>(c0, c, n), kQ<DT> - 1);
}
// acc += steps [s0, s1) as stream_run
template <int DT, int TRANS, int NG, int NF, int U, typename Fn>
__device__ __forceinline__ void cols_run(const ColsWeights<DT, TRANS, NF>& w, const StreamX<DT, 1, NG>& x, int s0,
                                         int s1, int kn, f32x4_t (&acc)[NF][NG], u32x4_t* scratch, int lane,
                                         Fn meanwhile) {
    constexpr int ST = kStep<DT>;
    const int full = min(s1, kn / ST);
    u32x4_t wa[U][NF], wb[U][NF], xa[U][NG][1], xb[U][NG][1];
    const auto load = [&](u32x4_t (&tw)[U][NF], u32x4_t (&tx)[U][NG][1], int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            w.load(tw[u], (s + u) * ST);
            x.load(tx[u], (s + u) * ST);
        }
    };
    const auto mul1 = [&](u32x4_t (&tw)[NF], const u32x4_t (&tx)[NG][1]) {
        u32x4_t o[NG][1];
        x.operands(tx, o, scratch, lane);
        if constexpr (TRANS)
            row_tile<NF>(tw, scratch, lane);
        else
            w.operands(tw, scratch, lane);
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if constexpr (DT == 2) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[j][g] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            __uint_as_float(tw[j][t]), __uint_as_float(o[g][0][t]), acc[j][g], 0, 0, 0);
                } else {
                    acc[j][g] = mfma16x16x32<DT>(tw[j], o[g][0], acc[j][g]);
                }
            }
    };
    const auto mul = [&](u32x4_t (&tw)[U][NF], const u32x4_t (&tx)[U][NG][1]) {
#pragma unroll
        for (int u = 0; u < U; ++u) mul1(tw[u], tx[u]);
    };
    int s = s0;
    if (s + U <= full) load(wa, xa, s);
    meanwhile();
    for (; s + 2 * U <= full; s += 2 * U) {
        load(wb, xb, s + U);
        mul(wa, xa);
        if (s + 3 * U <= full) load(wa, xa, s + 2 * U);
        mul(wb, xb);
    }
    if (s + U <= full) {
        mul(wa, xa);
        s += U;
    }
    for (; s < s1 && s * ST < kn; ++s) {  // the rest, the last step with zeros past kn
        w.tail(wa[0], s * ST, kn, lane);
        x.tail(xa[0], s * ST, kn, lane);
        mul1(wa[0], xa[0]);
    }
}

// ------------------------------------------------------------------ parts of one result in several workgroups
// A workgroup leaves its part of a row's CW columns in parts[row][CW], past
// its own L2 (another one's workgroup may sum it), and counts itself; the last
// one of a column block to be counted sums the parts.  Whole lines
// belong to one column block, and they are read with loads that do not look
// into this L2 either, so no cache has to be invalidated.
template <int CW>
__device__ __forceinline__ void part_store(float* parts, int64_t row, int c, float v) {
    __hip_atomic_store(parts + row * CW + c, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// whether this workgroup is the last of `count` (every thread calls it)
__device__ __forceinline__ bool part_last(uint32_t* done, uint32_t count, int tid) {
    __shared__ int last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores have reached memory
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == count - 1;
    __syncthreads();
    return last != 0;
}
// Calls out(m, c, v0, v1) with the sums over p in [0, np) of parts[first(m) +
// step(p)][c], [c + 1] for the M rows and CW / 2 column pairs; a thread has NB * SB
// loads on their way at once (a round trip to memory takes as long as all of
// them).  The order of the sum is fixed.
template <int NT, int CW, int NB, int SB, typename Row, typename Out>
__device__ __forceinline__ void part_sums(const float* parts, int M, int np, int tid, Row row, Out out) {
    for (int o0 = tid; o0 < M * (CW / 2); o0 += NT * NB) {
        float v[NB][2] = {};
        for (int p0 = 0; p0 < np; p0 += SB) {
            uint64_t u[NB][SB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int o = min(o0 + b * NT, M * (CW / 2) - 1);
#pragma unroll
                for (int i = 0; i < SB; ++i)
                    u[b][i] = __hip_atomic_load(
                        (const uint64_t*)(parts + row(o / (CW / 2), min(p0 + i, np - 1)) * CW + o % (CW / 2) * 2),
                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < SB; ++i)
                    if (p0 + i < np) {
                        v[b][0] += __uint_as_float((uint32_t)u[b][i]);
                        v[b][1] += __uint_as_float((uint32_t)(u[b][i] >> 32));
                    }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int o = o0 + b * NT;
            if (o < M * (CW / 2)) out(o / (CW / 2), o % (CW / 2) * 2, v[b][0], v[b][1]);
        }
    }
}
template <int NT, int CW, typename Row, typename Out>
__device__ __forceinline__ void part_sums(const float* parts, int M, int np, int tid, Row row, Out out) {
    if (M * (CW / 2) <= NT)
        part_sums<NT, CW, 1, 16>(parts, M, np, tid, row, out);
    else
        part_sums<NT, CW, 4, 8>(parts, M, np, tid, row, out);
}

}  // namespace omm
