// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits, in one pass over them, and the gradient.
//
// Per row x[0..V):  m = max x,  s = sum e^(x-m),  t = sum e^(x-m) (x-m):
//   lse = m + ln s,  logprob = (x[target] - m) - ln s,  entropy = ln s - t / s.
// All three are kept online: a new maximum m' = m + d rescales s by e^-d and
// turns t into e^-d (t - d s).  (t and d are held in units of log2.)
//
// The k largest come from the same pass: a lane keeps the three largest of its
// vectors' maxima and where they were.  The k-th largest of the workgroup's
// lane maxima is a lower bound T of the row part's k-th largest element (values
// and indices are ordered together, so equal values need no case of their own).
// A lane reads its first two vectors again if they reach T, and all of its
// elements only if the third does (with 20 of 50001 tokens: about one lane a
// row); what reaches T is listed and ranked by (value, lower index).  Without
// the positions every lane that reached T read all of its elements again, as
// many cache lines as the row has: 2048 rows of 50001, 20 alternatives, 73 us;
// now 52, of which the first pass is 38 without positions (5.4 TB/s, the vector
// ALU about as busy) and 43 with them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"
#include "row_select.hpp"

namespace omm {

namespace {

constexpr int kTopMax = 32;      // top_k bound (checked by the caller)
constexpr int kCand = 1024;      // candidates that fit the list; more go by rounds
constexpr int kSplitMax = 64;    // row parts; one lane of the join each
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

struct Stat {
    float m, s, t;
};

// 2^((a-b) log2 e) with a <= b; a = -inf gives 0 for any b
__device__ __forceinline__ float d_log2(float a, float b) { return (a - b) * kLog2e; }

// Finite stand-in for a running maximum of -inf (nothing but -inf so far):
// x - 0 = -inf, whose exponential is 0, where -inf - -inf would be NaN.
__device__ __forceinline__ float safe_max(float m) { return m == kNegInf ? 0.0f : m; }

__device__ __forceinline__ Stat merge(Stat a, Stat b) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    const float ms = safe_max(r.m);
    const float da = d_log2(a.m, ms), db = d_log2(b.m, ms);
    const float ea = __builtin_amdgcn_exp2f(da), eb = __builtin_amdgcn_exp2f(db);
    r.s = a.s * ea + b.s * eb;
    // a part that is all -inf has t = s = 0; the clamp keeps 0 * -inf out
    r.t = ea * (a.t + a.s * fmaxf(da, -200.0f)) + eb * (b.t + b.s * fmaxf(db, -200.0f));
    return r;
}

// The three largest of a lane's positions (a head element, vectors in order, a
// tail element) by order key; 0: none.  Positions come in ascending order, so
// of equal keys the first one is kept first.
struct Top3 {
    uint32_t k1, k2, k3;
    int b1, b2, b3;
    __device__ __forceinline__ void insert(uint32_t x, int pos) {
        const bool g1 = x > k1, g2 = x > k2;
        b3 = g2 ? b2 : x > k3 ? pos : b3;
        k3 = max(min(x, k2), k3);
        b2 = g1 ? b1 : g2 ? pos : b2;
        k2 = max(min(x, k1), k2);
        b1 = g1 ? pos : b1;
        k1 = max(x, k1);
    }
};

template <int N, bool TOP>
__device__ __forceinline__ void update(Stat& st, const float* f, int pos, Top3& top) {
    float mv = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mv = fmaxf(mv, f[i]);
    if constexpr (TOP) top.insert(order_key_finite(mv), pos);
    if (mv > st.m) {
        const float d = d_log2(st.m, mv);  // -inf for the first finite value
        const float e = __builtin_amdgcn_exp2f(d);
        st.t = e * (st.t + st.s * fmaxf(d, -200.0f));
        st.s *= e;
        st.m = mv;
    }
    const float ms = safe_max(st.m);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // (d is rounded once, which puts a term off by |d| 2^-24 of itself: in the sums
        // that averages out.  Corrected as in the gradient, 2048 rows of 50001 take 59
        // us instead of 52, and the error of 64 rows of 131072 stays at 4e-7.)
        const float d = (f[i] - ms) * kLog2e;
        const float e = __builtin_amdgcn_exp2f(d);  // NaN and +inf - +inf reach s
        st.s += e;
        st.t = fmaf(e, fmaxf(d, -200.0f), st.t);  // e = 0 below -200
    }
}

// One row part [v0, v1) seen by NT threads: an unaligned head of < kVec
// elements (one a thread), whole 16-byte vectors, a tail (one a thread).
template <int DT>
struct Part {
    typedef typename elem_of<DT>::type E;
    const E* row;
    int v0, v1;    // element range
    int head, nv;  // head elements, vectors
    __device__ __forceinline__ Part(const E* r, int a, int b) : row(r), v0(a), v1(b) {
        const int mis = (int)(((uintptr_t)(r + a) & 15) / sizeof(E));
        head = mis ? min(kVec<DT> - mis, b - a) : 0;
        nv = (b - a - head) / kVec<DT>;
    }
    __device__ __forceinline__ int tail0() const { return v0 + head + nv * kVec<DT>; }
    __device__ __forceinline__ u32x4_t vec(int j) const {
        return *(const u32x4_t*)(row + v0 + head + (int64_t)j * kVec<DT>);
    }
};

// first and last index of a lane's position: -1 its head element, 0 .. nv - 1 a
// vector, nv its tail element
template <int DT>
__device__ __forceinline__ int pos_first(const Part<DT>& p, int tid, int pos) {
    return pos < 0 ? p.v0 + tid : pos < p.nv ? p.v0 + p.head + pos * kVec<DT> : p.tail0() + tid;
}
template <int DT>
__device__ __forceinline__ int pos_last(const Part<DT>& p, int tid, int pos) {
    return pos_first(p, tid, pos) + (pos >= 0 && pos < p.nv ? kVec<DT> - 1 : 0);
}
// Calls f(value, index) for the elements of a position
template <int DT, typename F>
__device__ __forceinline__ void for_pos(const Part<DT>& p, int tid, int pos, F f) {
    const int v = pos_first(p, tid, pos);
    if (pos >= 0 && pos < p.nv) {
        float x[kVec<DT>];
        unpack16<DT>(p.vec(pos), x);
#pragma unroll
        for (int i = 0; i < kVec<DT>; ++i) f(x[i], v + i);
    } else {
        f(elem_f32<DT>(p.row[v]), v);
    }
}
// Calls f(value, index) for every element that thread `tid` of NT owns
template <int DT, int NT, typename F>
__device__ __forceinline__ void for_own(const Part<DT>& p, int tid, F f) {
    if (tid < p.head) f(elem_f32<DT>(p.row[p.v0 + tid]), p.v0 + tid);
    for (int j = tid; j < p.nv; j += NT) {
        float x[kVec<DT>];
        unpack16<DT>(p.vec(j), x);
#pragma unroll
        for (int i = 0; i < kVec<DT>; ++i) f(x[i], p.v0 + p.head + j * kVec<DT> + i);
    }
    const int q = p.tail0() + tid;
    if (q < p.v1) f(elem_f32<DT>(p.row[q]), q);
}

// Outputs of a row (splits == 1) or of a row part (ws)
struct LpArgs {
    const void* logits;
    const void* targets;  // int32 / int64
    float* logprobs;
    float* entropy;  // or nullptr
    float* lse;      // or nullptr
    int32_t* top_ids;
    float* top_lp;
    // parts: stats (m, s, t, 0) per (row, split), then k keys each
    float4* part_stat;
    uint64_t* part_key;
    int64_t M;
    int V, k, splits, chunk, idx64;
};

__device__ __forceinline__ int64_t load_target(const LpArgs& a, int64_t m) {
    return a.idx64 ? ((const int64_t*)a.targets)[m] : (int64_t)((const int32_t*)a.targets)[m];
}

// lse, entropy and the target's log probability of a whole row
template <int DT>
__device__ __forceinline__ void write_row(const LpArgs& a, int64_t m, Stat st, float log_s) {
    const typename elem_of<DT>::type* row = (const typename elem_of<DT>::type*)a.logits + m * (int64_t)a.V;
    const int64_t t = load_target(a, m);
    const bool empty = st.m == kNegInf && st.s == 0.0f;  // every logit is -inf
    float lp = 0.0f;  // a target outside [0, V) is ignored
    if (t >= 0 && t < a.V) {
        const float x = elem_f32<DT>(row[t]);
        lp = empty ? kNegInf : (x - st.m) - log_s;
    }
    a.logprobs[m] = lp;
    if (a.lse) a.lse[m] = empty ? kNegInf : st.m + log_s;
    if (a.entropy) a.entropy[m] = empty ? 0.0f : log_s - st.t * kLn2 / st.s;
}

__device__ __forceinline__ float top_logprob(uint64_t key, Stat st, float log_s) {
    if (st.s != st.s) return st.s;  // a NaN in the row
    const float x = key_value((uint32_t)(key >> 32));
    return x == kNegInf ? kNegInf : (x - st.m) - log_s;
}

// The k-th largest of a wave's lane maxima as one key: value T, and the largest
// index I up to which elements of value T count (ties go to the lower index).
// A bit a step from the top.  16 bits of the value will do, a lower T only
// lists more; the index is looked for where many lanes have T itself.  `idx` is
// the last index of the maximum's position (so each of the k lanes has an
// element that counts).
__device__ __forceinline__ uint64_t kth_lane(uint32_t x, int idx, int k) {
    uint32_t T = 0;
    int count = 64;  // lanes >= T
    for (int b = 31; b >= 16; --b) {
        const uint32_t c = T | (1u << b);
        const int n = __popcll(__ballot(x >= c));
        if (n >= k) {
            T = c;
            count = n;
        }
    }
    if (count <= k + 16) return order_key64(T, 0x7fffffffu);
    for (int b = 15; b >= 0; --b) {
        const uint32_t c = T | (1u << b);
        if (__popcll(__ballot(x >= c)) >= k) T = c;
    }
    const int more = k - __popcll(__ballot(x > T));
    const int v = x == T ? idx : 0x7fffffff;
    int lim = 0;  // the more-th smallest index: the largest lim with fewer below it
    for (int b = 30; b >= 0; --b) {
        const int c = lim | (1 << b);
        if (__popcll(__ballot(v < c)) < more) lim = c;
    }
    return order_key64(T, (uint32_t)lim);
}

template <int DT, int NT, bool TOP>
__global__ __launch_bounds__(NT, 8) void logprobs_kernel(LpArgs a) {
    typedef typename elem_of<DT>::type E;
    constexpr int NW = NT / 64;
    __shared__ Stat sh_stat[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t m = blockIdx.x / a.splits;
    const int sp = (int)(blockIdx.x - m * a.splits);
    const int v0 = min(a.V, sp * a.chunk), v1 = min(a.V, v0 + a.chunk);
    const Part<DT> p((const E*)a.logits + m * (int64_t)a.V, v0, v1);

    Stat st = {kNegInf, 0.0f, 0.0f};
    Top3 top = {0, 0, 0, 0, 0, 0};
    if (tid < p.head) {
        const float f = elem_f32<DT>(p.row[p.v0 + tid]);
        update<1, TOP>(st, &f, -1, top);
    }
    for (int j = tid; j < p.nv; j += NT) {
        float x[kVec<DT>];
        unpack16<DT>(p.vec(j), x);
        update<kVec<DT>, TOP>(st, x, j, top);
    }
    if (p.tail0() + tid < p.v1) {
        const float f = elem_f32<DT>(p.row[p.tail0() + tid]);
        update<1, TOP>(st, &f, p.nv, top);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const Stat o = {__shfl_xor(st.m, d, 64), __shfl_xor(st.s, d, 64), __shfl_xor(st.t, d, 64)};
        st = merge(st, o);
    }
    if (lane == 0) sh_stat[wave] = st;
    if constexpr (!TOP) {
        __syncthreads();
        st = sh_stat[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) st = merge(st, sh_stat[w]);
    } else {
        __shared__ uint64_t sh_bound[NW];
        __shared__ uint64_t sh_cand[kCand + 8];  // (zeros after the last one)
        __shared__ uint64_t sh_red[NW];
        __shared__ uint64_t sh_top[kTopMax];
        __shared__ int sh_n;
        // (a wave has 64 maxima; fewer elements than k: all are listed)
        const uint64_t bound = kth_lane(top.k1, pos_last(p, tid, top.b1), a.k);
        if (lane == 0) sh_bound[wave] = bound;
        if (tid == 0) sh_n = 0;
        __syncthreads();
        st = sh_stat[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) st = merge(st, sh_stat[w]);
        const bool nan_row = st.s != st.s;  // NaN is above every value, fmaxf has not seen it
        int n = kCand + 1;
        if (!nan_row) {
            uint64_t best = sh_bound[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) best = sh_bound[w] > best ? sh_bound[w] : best;
            const uint32_t T = (uint32_t)(best >> 32);
            const int I = (int)key64_index(best);
            const auto list = [&](float x, int v) {
                const uint32_t key = order_key(x);
                if (key > T || (key == T && v <= I)) {
                    const int i = atomicAdd(&sh_n, 1);
                    if (i < kCand) sh_cand[i] = order_key64(key, (uint32_t)v);
                }
            };
            // (key 0: no element; T = 0 where fewer than k lanes have one)
            const auto reaches = [&](uint32_t key, int first) { return key > T || (key == T && key && first <= I); };
            const bool one = reaches(top.k1, pos_first(p, tid, top.b1));
            const bool two = reaches(top.k2, pos_first(p, tid, top.b2));
            // (what comes after the third position in this order cannot reach if it does not)
            const bool all = reaches(top.k3, pos_first(p, tid, top.b3));
            if (one && !all) for_pos(p, tid, top.b1, list);
            if (two && !all) for_pos(p, tid, top.b2, list);
            // all of a lane's elements: the wave reads them, a vector a lane
            for (uint64_t todo = __ballot(all); todo; todo &= todo - 1) {
                const int t = wave * 64 + __ffsll((unsigned long long)todo) - 1;
                for (int j = t + NT * lane; j < p.nv; j += NT * 64) for_pos(p, t, j, list);
                if (lane == 0 && t < p.head) for_pos(p, t, -1, list);
                if (lane == 1 && p.tail0() + t < p.v1) for_pos(p, t, p.nv, list);
            }
            __syncthreads();
            n = sh_n;
        }
        const int kk = min(a.k, v1 - v0);
        if (n <= kCand) {  // rank the list: every key is of its own, so ranks are too
            if (tid < 8) sh_cand[n + tid] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += NT) {
                const uint64_t key = sh_cand[i];
                int r = 0;
                for (int j = 0; j < n; j += 8)
#pragma unroll
                    for (int u = 0; u < 8; ++u) r += sh_cand[j + u] > key;
                if (r < kk) sh_top[r] = key;
            }
            __syncthreads();
        } else {  // NaN, or more candidates than fit: the largest key below the last one, k times
            uint64_t last = ~0ull;
            for (int r = 0; r < kk; ++r) {
                uint64_t mx = 0;
                for_own<DT, NT>(p, tid, [&](float x, int v) {
                    const uint64_t key = order_key64(order_key(x), (uint32_t)v);
                    if (key < last && key > mx) mx = key;
                });
                mx = wave_max(mx);
                if (lane == 0) sh_red[wave] = mx;
                __syncthreads();
                mx = sh_red[0];
#pragma unroll
                for (int w = 1; w < NW; ++w) mx = sh_red[w] > mx ? sh_red[w] : mx;
                if (tid == 0) sh_top[r] = mx;
                last = mx;
                __syncthreads();
            }
        }
        if (tid < a.k) {
            const uint64_t key = tid < kk ? sh_top[tid] : 0;  // 0: the part has fewer than k elements
            if (a.splits > 1) {
                a.part_key[(m * a.splits + sp) * a.k + tid] = key;
            } else {
                a.top_ids[m * a.k + tid] = (int32_t)key64_index(key);
                a.top_lp[m * a.k + tid] = top_logprob(key, st, logf(st.s));
            }
        }
    }
    if (tid == 0) {
        if (a.splits > 1)
            a.part_stat[m * a.splits + sp] = make_float4(st.m, st.s, st.t, 0.0f);
        else
            write_row<DT>(a, m, st, logf(st.s));
    }
}

// One workgroup a row joins its parts.  Up to 256 keys are ranked, one a thread;
// of more, as each part's are in descending order, lane i of the first wave
// holds part i and the k largest are k rounds of "largest head, advance".  (300
// rows of 4 parts, 20 keys each: rounds 7.2 us, ranked by one wave 5.1.)
template <int DT>
__global__ __launch_bounds__(256) void logprobs_join_kernel(LpArgs a) {
    __shared__ uint64_t keys[kSplitMax * kTopMax + 8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t m = blockIdx.x;
    Stat st = {kNegInf, 0.0f, 0.0f};
    if (lane < a.splits) {
        const float4 v = a.part_stat[m * a.splits + lane];
        st = {v.x, v.y, v.z};
    }
    const int n = a.splits * a.k;
    for (int i = tid; i < n; i += 256) keys[i] = a.part_key[m * n + i];
    if (tid < 8) keys[n + tid] = 0;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const Stat o = {__shfl_xor(st.m, d, 64), __shfl_xor(st.s, d, 64), __shfl_xor(st.t, d, 64)};
        st = merge(st, o);
    }
    const float log_s = logf(st.s);
    if (tid == 0) write_row<DT>(a, m, st, log_s);
    if (n == 0) return;
    __syncthreads();
    if (n <= 256) {
        if (tid >= n) return;
        const uint64_t own = keys[tid];
        int rank = 0;
        for (int j = 0; j < n; j += 8)
#pragma unroll
            for (int u = 0; u < 8; ++u) rank += keys[j + u] > own;
        if (own && rank < a.k) {
            a.top_ids[m * a.k + rank] = (int32_t)key64_index(own);
            a.top_lp[m * a.k + rank] = top_logprob(own, st, log_s);
        }
        return;
    }
    if (tid >= 64) return;
    int h = 0;
    uint64_t head = lane < a.splits ? keys[lane * a.k] : 0, mine = 0;
    for (int r = 0; r < a.k; ++r) {
        // (value, then index: two 32-bit maxima by DPP)
        const uint32_t hi = wave_max_u32((uint32_t)(head >> 32));
        const uint32_t lo = wave_max_u32((uint32_t)(head >> 32) == hi ? (uint32_t)head : 0);
        const uint64_t mx = ((uint64_t)hi << 32) | lo;
        if (lane == r) mine = mx;
        if (head == mx) head = ++h < a.k ? keys[lane * a.k + h] : 0;  // keys are distinct: one lane
    }
    if (lane < a.k) {
        a.top_ids[m * a.k + lane] = (int32_t)key64_index(mine);
        a.top_lp[m * a.k + lane] = top_logprob(mine, st, log_s);
    }
}

struct LpGradArgs {
    const void* logits;
    const void* targets;
    const float* lse;
    const float* entropy;     // or nullptr
    const float* g_logprobs;
    const float* g_entropy;   // or nullptr
    void* dlogits;
    int64_t M;
    int V, chunks, chunk, idx64;
};

// dx[v] = gl ([v = target] - p) - gH p (ln p + H),  p = e^(x - lse)
// One read and one write: 4096 rows of 131072 (bf16) in 380 us, 5.6 TB/s.
template <int DT>
struct GradRow {
    float gl, gh, H, lse;
    int t;
    __device__ __forceinline__ float operator()(float x, int v) const {
        // p = 0 below -200: the clamp keeps 0 * -inf (a masked logit) out
        const float l = x - lse, lc = fmaxf(l, -200.0f), b = l * kLog2e;
        float p = __builtin_amdgcn_exp2f(b);
        // What the rounding of b leaves of l: without it p would be off by |l| 2^-24.
        // Only a fp32 gradient shows it (131 rows of 55296 in bf16: 7.3 us with it, 6.8 without).
        if constexpr (DT == 2) p = fmaf(p, fmaf(fmaxf(b, -200.0f * kLog2e), -kLn2, lc), p);
        float d = -p * fmaf(gh, lc + H, gl);
        return v == t ? d + gl : d;
    }
};

template <int DT, int NT>
__global__ __launch_bounds__(NT) void logprobs_grad_kernel(LpGradArgs a) {
    typedef typename elem_of<DT>::type E;
    const int tid = threadIdx.x;
    const int64_t m = blockIdx.x / a.chunks;
    const int c = (int)(blockIdx.x - m * a.chunks);
    const int v0 = min(a.V, c * a.chunk), v1 = min(a.V, v0 + a.chunk);
    const E* row = (const E*)a.logits + m * (int64_t)a.V;
    E* out = (E*)a.dlogits + m * (int64_t)a.V;
    GradRow<DT> g;
    const int64_t t = a.idx64 ? ((const int64_t*)a.targets)[m] : (int64_t)((const int32_t*)a.targets)[m];
    g.t = t >= 0 && t < a.V ? (int)t : -1;
    g.gl = g.t >= 0 ? a.g_logprobs[m] : 0.0f;
    g.gh = a.g_entropy ? a.g_entropy[m] : 0.0f;
    g.H = a.g_entropy ? a.entropy[m] : 0.0f;
    g.lse = a.lse[m];
    if (g.lse == kNegInf) {  // every logit is -inf: p = 0 everywhere
        g.gl = g.gh = g.H = g.lse = 0.0f;
    }
    const Part<DT> p(row, v0, v1);
    // logits and gradient are stored alike, but may start at different alignments
    const bool vec_out = (((uintptr_t)(out + v0 + p.head)) & 15) == 0;
    if (tid < p.head) out[v0 + tid] = f32_elem<DT>(g(elem_f32<DT>(row[v0 + tid]), v0 + tid));
    for (int j = tid; j < p.nv; j += NT) {
        float x[kVec<DT>];
        unpack16<DT>(p.vec(j), x);
        const int v = v0 + p.head + j * kVec<DT>;
#pragma unroll
        for (int i = 0; i < kVec<DT>; ++i) x[i] = g(x[i], v + i);
        if (vec_out) {
            u32x4_t o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == 2)
                    o[i] = __float_as_uint(x[i]);
                else
                    o[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
            }
            *(u32x4_t*)(out + v) = o;
        } else {
#pragma unroll
            for (int i = 0; i < kVec<DT>; ++i) out[v + i] = f32_elem<DT>(x[i]);
        }
    }
    const int q = p.tail0() + tid;
    if (q < v1) out[q] = f32_elem<DT>(g(elem_f32<DT>(row[q]), q));
}

// Row parts: enough workgroups to fill the chip when there are few rows, but
// no part under 4096 elements, and rows of up to 16384 whole: the second kernel
// costs more than their other parts would save (1 row of 16000, bf16, 10.0 us in
// 4 parts, 7.8 whole; of 32000 9.9 and 10.4).
void plan_splits(int64_t M, int64_t V, int* splits, int* chunk) {
    int64_t s = 1;
    if (M < 512) s = (1024 + M - 1) / M;
    const int64_t most = (V + 4095) / 4096;
    if (s > most) s = most;
    if (V <= 16384) s = 1;
    if (s > kSplitMax) s = kSplitMax;
    if (s < 1) s = 1;
    int64_t c = (V + s - 1) / s;
    c = (c + 63) / 64 * 64;
    *chunk = (int)c;
    *splits = (int)((V + c - 1) / c);
}

}  // namespace

size_t token_logprobs_workspace_bytes(int64_t M, int64_t V, int64_t k) {
    if (M <= 0 || V <= 0) return 0;
    int splits, chunk;
    plan_splits(M, V, &splits, &chunk);
    if (splits <= 1) return 0;
    return (size_t)M * splits * (16 + 8 * (size_t)k);
}

hipError_t launch_token_logprobs(const TokenLogprobsArgs& t, int dt, void* ws, hipStream_t s) {
    LpArgs a;
    a.logits = t.logits;
    a.targets = t.targets;
    a.logprobs = t.logprobs;
    a.entropy = t.entropy;
    a.lse = t.lse;
    a.top_ids = t.top_ids;
    a.top_lp = t.top_logprobs;
    a.M = t.M;
    a.V = (int)t.V;
    a.k = t.k;
    a.idx64 = t.idx64;
    plan_splits(t.M, t.V, &a.splits, &a.chunk);
    a.part_stat = (float4*)ws;
    a.part_key = (uint64_t*)((char*)ws + (size_t)t.M * a.splits * 16);
    log_choice("token_logprobs: %d part(s) of %d a row", a.splits, a.chunk);
    const dim3 grid((unsigned)(t.M * a.splits));
    switch (dt * 2 + (a.k > 0)) {
        case 0: logprobs_kernel<0, 256, false><<<grid, 256, 0, s>>>(a); break;
        case 1: logprobs_kernel<0, 256, true><<<grid, 256, 0, s>>>(a); break;
        case 2: logprobs_kernel<1, 256, false><<<grid, 256, 0, s>>>(a); break;
        case 3: logprobs_kernel<1, 256, true><<<grid, 256, 0, s>>>(a); break;
        case 4: logprobs_kernel<2, 256, false><<<grid, 256, 0, s>>>(a); break;
        default: logprobs_kernel<2, 256, true><<<grid, 256, 0, s>>>(a); break;
    }
    if (a.splits > 1) {
        const dim3 jg((unsigned)t.M);
        if (dt == 0) logprobs_join_kernel<0><<<jg, 256, 0, s>>>(a);
        else if (dt == 1) logprobs_join_kernel<1><<<jg, 256, 0, s>>>(a);
        else logprobs_join_kernel<2><<<jg, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_token_logprobs_grad(const TokenLogprobsGradArgs& t, int dt, hipStream_t s) {
    LpGradArgs a;
    a.logits = t.logits;
    a.targets = t.targets;
    a.lse = t.lse;
    a.entropy = t.entropy;
    a.g_logprobs = t.g_logprobs;
    a.g_entropy = t.g_entropy;
    a.dlogits = t.dlogits;
    a.M = t.M;
    a.V = (int)t.V;
    a.idx64 = t.idx64;
    // workgroups of 16384 elements, of fewer where that leaves the chip unfilled
    // (64 rows of 32000 fp32: 7.1 us in 128 workgroups, 4.3 in 1024)
    a.chunk = 16384;
    while (a.chunk > 2048 && t.M * ((t.V + a.chunk - 1) / a.chunk) < 1024) a.chunk /= 2;
    a.chunks = (int)((t.V + a.chunk - 1) / a.chunk);
    const dim3 grid((unsigned)(t.M * a.chunks));
    if (dt == 0) logprobs_grad_kernel<0, 256><<<grid, 256, 0, s>>>(a);
    else if (dt == 1) logprobs_grad_kernel<1, 256><<<grid, 256, 0, s>>>(a);
    else logprobs_grad_kernel<2, 256><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace omm
