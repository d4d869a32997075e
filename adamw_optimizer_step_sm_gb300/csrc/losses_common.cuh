// losses_common.cuh -- device building blocks of the fine-tuning operators:
// element types, 16-byte vectors, the online softmax record and its joins, the
// error-free running sum, cluster access, token weights and the policy loss of
// one token; and the host helpers of their entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>

#include "adamw_internal.h"
#include "adamw_losses.h"

// Internal linkage, as in device_common.cuh.
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = std::numeric_limits<float>::infinity();
constexpr float kMaxFloat = std::numeric_limits<float>::max();

// ------------------------------------------------------- pairs of floats --

// Two floats in a 64-bit register, for the packed fp32 instructions (sm_100
// and later): one instruction does both.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float low(Pair p) { return __uint_as_float(uint32_t(p)); }
__device__ __forceinline__ float high(Pair p) { return __uint_as_float(uint32_t(p >> 32)); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Exponents that vanish all the same, to one whose product with the vanished
// exponential is 0 (not 0 * inf) and stays finite times a gradient; NaN to itself
// or to that number (its exponential is NaN already).
constexpr float kVanished = -1e4f;
__device__ __forceinline__ Pair above(Pair d) { return pair(fmaxf(low(d), kVanished), fmaxf(high(d), kVanished)); }

// A 32-bit register as two 16-bit floats.
template <typename T>
__device__ __forceinline__ T word(uint32_t w) {
    T t;
    memcpy(&t, &w, 4);
    return t;
}

// ------------------------------------------------------- element types ----

template <int DT>
struct Elem;

template <>
struct Elem<ADAMW_DTYPE_BF16> {
    static constexpr int kSize = 2, kVec = 8;
    static constexpr uint32_t kNegInf = 0xff80ff80u;   // two elements of -inf
    static constexpr uint32_t kSigns = 0x80008000u;
    __device__ static float load(const void* p, int64_t i) {
        return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
    }
    __device__ static void store(void* p, int64_t i, float x) {
        static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    }
    __device__ static void unpack(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            memcpy(&w[i], &r, 4);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the vector as pairs of floats; the largest element of some vectors
    __device__ static void pairs(uint4 v, Pair* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    template <int U>
    __device__ static float largest(const uint4 (&v)[U]) {
        __nv_bfloat162 m = word<__nv_bfloat162>(v[0].x);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m = __hmax2(m, __hmax2(word<__nv_bfloat162>(v[u].x), word<__nv_bfloat162>(v[u].y)));
            m = __hmax2(m, __hmax2(word<__nv_bfloat162>(v[u].z), word<__nv_bfloat162>(v[u].w)));
        }
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ static uint4 pack_pairs(const Pair* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 r = __floats2bfloat162_rn(low(x[i]), high(x[i]));
            memcpy(&w[i], &r, 4);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Elem<ADAMW_DTYPE_FP16> {
    static constexpr int kSize = 2, kVec = 8;
    static constexpr uint32_t kNegInf = 0xfc00fc00u;
    static constexpr uint32_t kSigns = 0x80008000u;
    __device__ static float load(const void* p, int64_t i) {
        return __half2float(static_cast<const __half*>(p)[i]);
    }
    __device__ static void store(void* p, int64_t i, float x) {
        static_cast<__half*>(p)[i] = __float2half_rn(x);
    }
    __device__ static void unpack(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 h;
            memcpy(&h, &w[i], 4);
            const float2 f = __half22float2(h);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ static uint4 pack(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 r = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            memcpy(&w[i], &r, 4);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static void pairs(uint4 v, Pair* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(word<__half2>(w[i]));
            x[i] = pair(f.x, f.y);
        }
    }
    template <int U>
    __device__ static float largest(const uint4 (&v)[U]) {
        __half2 m = word<__half2>(v[0].x);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m = __hmax2(m, __hmax2(word<__half2>(v[u].x), word<__half2>(v[u].y)));
            m = __hmax2(m, __hmax2(word<__half2>(v[u].z), word<__half2>(v[u].w)));
        }
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ static uint4 pack_pairs(const Pair* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 r = __floats2half2_rn(low(x[i]), high(x[i]));
            memcpy(&w[i], &r, 4);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Elem<ADAMW_DTYPE_FP32> {
    static constexpr int kSize = 4, kVec = 4;
    static constexpr uint32_t kNegInf = 0xff800000u;
    static constexpr uint32_t kSigns = 0x80000000u;
    __device__ static float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    __device__ static void store(void* p, int64_t i, float x) { static_cast<float*>(p)[i] = x; }
    __device__ static void unpack(uint4 v, float* x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    __device__ static uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    __device__ static void pairs(uint4 v, Pair* x) {
        x[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    template <int U>
    __device__ static float largest(const uint4 (&v)[U]) {
        float m = __uint_as_float(v[0].x);
#pragma unroll
        for (int u = 0; u < U; ++u)
            m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[u].x)), fmaxf(__uint_as_float(v[u].y), __uint_as_float(v[u].z))),
                      __uint_as_float(v[u].w));
        return m;
    }
    __device__ static uint4 pack_pairs(const Pair* x) {
        return make_uint4(__float_as_uint(low(x[0])), __float_as_uint(high(x[0])), __float_as_uint(low(x[1])),
                          __float_as_uint(high(x[1])));
    }
};

__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ void store16(void* p, uint4 v) { *static_cast<uint4*>(p) = v; }

// 2^x, results below the smallest normal number flushed to 0 (a probability
// that small is 0 in every output type but fp32, where it is below 1.2e-38).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Programmatic dependent launch: every kernel here is launched with the
// attribute, reads nothing before the wait and lets the next kernel of the
// stream be set up from its start (it waits in turn).
__device__ __forceinline__ void dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependency_trigger() {
    asm volatile("griddepcontrol.launch_dependents;");
}

// -------------------------------------------------------------- clusters --

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// A barrier of every thread of the cluster; memory written before it is
// visible to the cluster after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
// The float at the same shared address in the cluster's CTA `rank`.
__device__ __forceinline__ float load_remote(const float* smem, uint32_t rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    float v;
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [ra];\n\t}"
                 : "=f"(v) : "r"(a), "r"(rank) : "memory");
    return v;
}

// ------------------------------------------------- error-free running sum --

// hi + lo, the rounding error of every addition found exactly (Knuth's TwoSum)
// and kept in lo: about 46 bits, at fp32's speed (fp64 additions are slow on
// this GPU).  A non-finite term makes hi or lo non-finite; value() is then
// NaN or the infinity.
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x);
        const float b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
        hi = s;
    }
    __device__ __forceinline__ void join(float h, float l) {
        add(h);
        lo = __fadd_rn(lo, l);
    }
    __device__ __forceinline__ float value() const {
        return isfinite(hi) ? __fadd_rn(hi, lo) : hi;
    }
};

// Sum over the warp, the same in every lane.
__device__ __forceinline__ Sum2 warp_sum(Sum2 a) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, a.hi, d);
        const float l = __shfl_xor_sync(0xffffffffu, a.lo, d);
        // both lanes add in the same order, so that they agree bit for bit
        const bool low = (threadIdx.x & d) == 0;
        Sum2 s = low ? a : Sum2{h, l};
        s.join(low ? h : a.hi, low ? l : a.lo);
        a = s;
    }
    return a;
}

// -------------------------------------------------------- online softmax --

// Exponentials are taken in base 2: with c = scale log2(e), exp(scale x) is
// 2^(c x).  Over the elements x seen so far, m is their largest, and
//     s = sum 2^(c x - r),  t = sum 2^(c x - r) (c x - r)  (for the entropy)
// with r = c m as rounded to fp32, so that each exponent is one fused
// multiply-add, rounded once.  -inf elements (and an empty record) leave m at
// -inf and add nothing; r is then 0, so that -inf - (-inf) does not arise.
// The largest element's own exponent is what r was rounded by: up to 32 where
// |c m| < 2^30.  Beyond that ("extreme": masks by large finite numbers) it soon
// leaves fp32's range, but there neighbouring floats are 64 and more apart in
// the exponent: nothing below such a maximum counts beside it.  So a record
// with an extreme maximum holds no sums (s is NaN where it saw a NaN, else
// unspecified); they are dropped when a larger element comes, and a row whose
// largest element is extreme counts the elements equal to it (row_join).
struct Online {
    float m, s, t;
};

__device__ __forceinline__ bool extreme(float m, float c) { return m != -kInf && !(fabsf(m) * c < 0x1p30f); }
// Rounded in every use alike: the compiler may not fuse the product into an
// addition, where it would stay unrounded.  Not -inf where m is finite: a -inf
// element less that would be NaN.
__device__ __forceinline__ float reference(float m, float c) {
    return m == -kInf ? 0.0f : fmaxf(__fmul_rn(m, c), -kMaxFloat);
}

// The exponent of an element, whatever m.
__device__ __forceinline__ float exponent(float x, float m, float c) {
    return extreme(m, c) ? (x - m) * c : fmaf(x, c, -reference(m, c));
}

// Moves a record's reference to that of M >= o.m.
template <bool ENT>
__device__ __forceinline__ void rebase(Online& o, float M, float c) {
    if (o.m == M) return;
    if (o.m == -kInf) {   // s is 0, or NaN when it saw a NaN, which stays
        o.m = M;
        return;
    }
    if (extreme(o.m, c)) {
        o.s = o.s == o.s ? 0.0f : o.s;
        if (ENT) o.t = 0.0f;
        o.m = M;
        return;
    }
    const float d = fmaxf(__fsub_rn(reference(o.m, c), reference(M, c)), -1e30f);
    const float f = exp2_fast(d);
    // d f before s: both d s and f's smallness may pass fp32's range
    if (ENT) o.t = fmaf(d * f, o.s, o.t * f);
    o.s *= f;
    o.m = M;
}

template <bool ENT>
__device__ __forceinline__ void join(Online& a, Online b, float c) {
    const float M = fmaxf(a.m, b.m);
    rebase<ENT>(a, M, c);
    rebase<ENT>(b, M, c);
    a.s += b.s;
    if (ENT) a.t += b.t;
}

template <bool ENT>
__device__ __forceinline__ void absorb_one(Online& o, float x, float c) {
    if (x > o.m) rebase<ENT>(o, x, c);
    const float d = exponent(x, o.m, c);
    const float e = exp2_fast(d);
    o.s += e;
    if (ENT) o.t = fmaf(e, fmaxf(d, kVanished), o.t);
}

// Adds the elements of U vectors.
template <int DT, bool ENT, int U>
__device__ __forceinline__ void absorb(Online& o, const uint4 (&v)[U], float c) {
    using E = Elem<DT>;
    const float m = E::largest(v);
    if (m > o.m) rebase<ENT>(o, m, c);
    const float r = -reference(o.m, c);
    const Pair c2 = pair(c, c), r2 = pair(r, r);
    Pair s = pair(0.0f, 0.0f), t = s;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        Pair x[E::kVec / 2];
        E::pairs(v[u], x);
#pragma unroll
        for (int i = 0; i < E::kVec / 2; ++i) {
            const Pair d = fma2(x[i], c2, r2);
            const Pair e = pair(exp2_fast(low(d)), exp2_fast(high(d)));
            s = add2(s, e);
            if (ENT) t = fma2(e, above(d), t);
        }
    }
    o.s += low(s) + high(s);
    if (ENT) o.t += low(t) + high(t);
}

template <bool ENT>
__device__ __forceinline__ Online warp_join(Online o, float c) {
    float M = o.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    rebase<ENT>(o, M, c);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        o.s += __shfl_xor_sync(0xffffffffu, o.s, d);
        if (ENT) o.t += __shfl_xor_sync(0xffffffffu, o.t, d);
    }
    return o;
}

constexpr float kLn2 = 0.6931471805599453f;

// What a row's softmax comes to: m and s as in Online, with s = +inf for a
// row without a distribution, or not read.
struct RowStats {
    float m, s, log_s, entropy;
};

template <bool ENT>
__device__ __forceinline__ RowStats row_stats(const Online& o) {
    if (o.m == -kInf && o.s == 0.0f) return {0.0f, kInf, kInf, 0.0f};
    const float log_s = logf(o.s);
    return {o.m, o.s, log_s, ENT ? log_s - kLn2 * (o.t / o.s) : 0.0f};
}

// log-probability of a logit x under the row.
__device__ __forceinline__ float logp_of(const RowStats& r, float x, float scale, float c) {
    if (r.s == kInf) return -kInf;
    const float d = exponent(x, r.m, c);
    // an exponent past fp32's range: the type's lowest value in an ordinary row,
    // or beside its largest (half the difference is a number of the type)
    return (d == -kInf ? (0.5f * x - 0.5f * r.m) * (2.0f * scale) : kLn2 * d) - r.log_s;
}

// The gradient of an element, without the target's term a:
//     -p (a + b (log p + H)) = 2^d (A + B d),  d its exponent,
//     a = scale d_logp, b = scale d_entropy
struct Gradient {
    float m, c, A, B, a;
    bool extreme_row;
    __device__ __forceinline__ Gradient(float m, float s, float log_s, float c, float a, float b, float H)
        : m(m), c(c), A(-(a + b * (H - log_s)) / s), B(-b * kLn2 / s), a(a), extreme_row(extreme(m, c)) {}

    template <bool ENT>
    __device__ __forceinline__ float of(float x) const {
        const float d = exponent(x, m, c), e = exp2_fast(d);
        return ENT ? e * fmaf(B, fmaxf(d, kVanished), A) : e * A;
    }
    // of a vector of an ordinary row
    template <int DT, bool ENT>
    __device__ __forceinline__ uint4 of(uint4 v) const {
        using E = Elem<DT>;
        const float r = -reference(m, c);
        const Pair c2 = pair(c, c), r2 = pair(r, r), A2 = pair(A, A), B2 = pair(B, B);
        Pair x[E::kVec / 2];
        E::pairs(v, x);
#pragma unroll
        for (int i = 0; i < E::kVec / 2; ++i) {
            const Pair d = fma2(x[i], c2, r2);
            const Pair e = pair(exp2_fast(low(d)), exp2_fast(high(d)));
            x[i] = mul2(e, ENT ? fma2(B2, above(d), A2) : A2);
        }
        return E::pack_pairs(x);
    }
};

// ----------------------------------------------------------------- rows ----

// adamw_rows_t for a kernel: byte strides.
struct Rows {
    char* data;
    int64_t outer, row;
    uint32_t inner;
    __device__ __forceinline__ char* at(uint32_t r) const {
        const uint32_t o = r / inner;
        return data + int64_t(o) * outer + int64_t(r - o * inner) * row;
    }
};

// A row as a few leading elements up to the first 16-byte boundary, whole
// vectors, and a few trailing elements.
template <int DT>
struct RowSplit {
    int head, vecs, tail;
    __device__ __forceinline__ RowSplit(const char* row, int cols) {
        using E = Elem<DT>;
        const int off = int((16u - (uint32_t(reinterpret_cast<uintptr_t>(row)) & 15u)) & 15u) / E::kSize;
        head = off < cols ? off : cols;
        vecs = (cols - head) / E::kVec;
        tail = cols - head - vecs * E::kVec;
    }
};

// ----------------------------------------------------------------- tokens --

// adamw_tokens_t for a kernel.  Tokens count by a byte mask, or by their
// target (not `ignore`), or all.
struct Tokens {
    uint32_t n, sequences, length;  // length: of each, without offsets
    const int64_t* offsets;
    const uint8_t* mask;
    const int64_t* targets;
    int64_t ignore;

    // The sequence of token i, or -1 outside of them all.  With offsets by
    // bisection, which stays inside the array whatever it holds.
    __device__ __forceinline__ int32_t sequence(uint32_t i) const {
        if (!offsets) return int32_t(i / length);
        uint32_t lo = 0, hi = sequences;  // the last start <= i is in [lo, hi)
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (offsets[mid] <= int64_t(i)) lo = mid; else hi = mid;
        }
        return int64_t(i) >= offsets[lo] && int64_t(i) < offsets[lo + 1] ? int32_t(lo) : -1;
    }

    // How many of the sequences + 1 offsets are at or before token `base`, the
    // same for a whole warp, which calls together: each round the lanes probe
    // 32 points of what is left, so 2048 offsets take three loads.
    __device__ __forceinline__ uint32_t starts_until(uint32_t base) const {
        if (!offsets) return 0;
        const uint32_t lane = threadIdx.x % 32;
        uint32_t lo = 0, hi = sequences + 1;  // offsets[0, lo) <= base < offsets[hi, ..)
        while (lo < hi) {
            const uint32_t step = (hi - lo + 31) / 32;
            const uint32_t at = lo + lane * step;
            const bool below = at < hi && offsets[at] <= int64_t(base);
            // ascending offsets: the lanes below are the first ones
            const uint32_t k = __popc(__ballot_sync(0xffffffffu, below));
            if (k == 0) break;
            const uint32_t next = lo + k * step;
            lo = lo + (k - 1) * step + 1;
            hi = next < hi ? next : hi;
        }
        return lo;
    }

    // The sequences of the N tokens from `first` on, for every lane of a warp
    // that covers [base, base + 32 N), with lo = starts_until(base).  Called
    // by whole warps.
    template <int N>
    __device__ __forceinline__ void sequences_of(uint32_t lo, uint32_t base, uint32_t first, int32_t (&seq)[N]) const {
        if (!offsets) {
            uint32_t q = first / length, r = first - q * length;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                seq[j] = int32_t(q);
                if (++r == length) { r = 0; ++q; }
            }
            return;
        }
        // the offsets inside the warp's tokens, in the lanes
        const uint32_t at = lo + threadIdx.x % 32;
        const int64_t past = int64_t(base) + 32 * N;
        const int64_t mine = at <= sequences ? offsets[at] : past;
        const int count = __popc(__ballot_sync(0xffffffffu, mine < past));
        const int32_t near = int32_t(mine < past ? mine - base : 32 * N), me = int32_t(first - base);
#pragma unroll
        for (int j = 0; j < N; ++j) seq[j] = int32_t(lo) - 1;
        if (count < 32) {
            for (int k = 0; k < count; ++k) {
                const int32_t b = __shfl_sync(0xffffffffu, near, k);
#pragma unroll
                for (int j = 0; j < N; ++j) seq[j] += b <= me + j;
            }
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (seq[j] >= int32_t(sequences)) seq[j] = -1;
        } else {  // more sequences here than lanes
#pragma unroll
            for (int j = 0; j < N; ++j) seq[j] = first + j < n ? sequence(first + j) : -1;
        }
    }

    // Whether N neighbouring tokens are all of sequence `s`.  All are compared:
    // -1 stands on both sides of the sequences, so the ends may agree where
    // the middle differs.
    template <int N>
    __device__ __forceinline__ static bool all_of(const int32_t (&seq)[N], int32_t s) {
        bool same = true;
#pragma unroll
        for (int j = 0; j < N; ++j) same = same && seq[j] == s;
        return same;
    }

    // Which of the N <= 4 tokens from `first` on count, as bits.
    template <int N>
    __device__ __forceinline__ uint32_t counting(uint32_t first) const {
        const uint32_t left = first < n ? n - first : 0;
        uint32_t bits = left >= N ? (1u << N) - 1 : (1u << left) - 1;
        if (mask) {
            if (N == 4 && left >= 4 && (reinterpret_cast<uintptr_t>(mask) + first) % 4 == 0) {
                // bytes to 0 / 1, then their bits next to one another
                const uint32_t w = *reinterpret_cast<const uint32_t*>(mask + first);
                bits = ((__vcmpne4(w, 0) & 0x01010101u) * 0x01020408u) >> 24;
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j < int(left) && mask[first + j] == 0) bits &= ~(1u << j);
            }
        } else if (targets) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < int(left) && targets[first + j] == ignore) bits &= ~(1u << j);
        }
        return bits;
    }
};

// Token counts, in the workspace: tokens and non-empty sequences first, then
// each sequence's tokens.
struct Counts {
    uint32_t tokens, filled, ticket, pad_;
    uint32_t sequence[1];
};

// 1 / x for 1 <= x < 2^126, within an ulp.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The weight of a token of a sequence with `in_sequence` tokens that count.
__device__ __forceinline__ float token_weight(int32_t reduce, float inv_divisor, uint32_t tokens,
                                              uint32_t filled, uint32_t in_sequence) {
    if (reduce == ADAMW_REDUCE_FIXED) return inv_divisor;
    if (reduce == ADAMW_REDUCE_TOKEN) return reciprocal(float(tokens));
    return reciprocal(float(in_sequence) * float(filled));
}

// ------------------------------------------------------------ policy loss --

// adamw_policy_t with the thresholds of d = logp - old_logp worked out.
struct Policy {
    float r_low, r_high, d_low, d_high, dual, d_dual;  // d_dual +inf: off
    float kl_coef, entropy_coef, inv_divisor, grad_scale;
    int32_t kl, reduce, per_token;
};

struct PolicyToken {
    float pg, kl, off, old_kl, grad;
};

// exp(x) - 1 - x, from x and e = exp(x).  Below 0.7 by its series, whose terms
// after x^9 are together below 4e-8 of the first (x^10 / 10! is 3.2e-8 of x^2 / 2
// there); above, the subtraction loses no more than three bits.
__device__ __forceinline__ float exp_beyond_linear(float x, float e) {
    float s = 1.0f / 362880.0f;
    s = fmaf(s, x, 1.0f / 40320.0f);
    s = fmaf(s, x, 1.0f / 5040.0f);
    s = fmaf(s, x, 1.0f / 720.0f);
    s = fmaf(s, x, 1.0f / 120.0f);
    s = fmaf(s, x, 1.0f / 24.0f);
    s = fmaf(s, x, 1.0f / 6.0f);
    s = fmaf(s, x, 0.5f);
    const float far = (e - 1.0f) - fminf(x, kMaxFloat);   // not inf - inf
    return fabsf(x) < 0.7f ? s * x * x : far;
}

// The loss terms of one token and the derivative of pg + kl_coef KL with
// respect to its log-probability (weights left out).
__device__ __forceinline__ PolicyToken policy_token(const Policy& P, float logp, float old, bool has_ref,
                                                    float ref, float A) {
    PolicyToken o;
    const float d = logp - old;
    const float r = expf(d);
    // Outside [low, high] the clipped branch holds; inside, -A r is the larger
    // of the two: where r is past a limit there, it is past it on the side
    // that makes -A r larger.
    const bool up = A > 0.0f;
    const float high = up ? P.d_high : P.d_dual, low = up ? -kInf : P.d_low;
    const bool off = A != 0.0f && (d > high || d < low);
    const float bound = up ? P.r_high : d < low ? P.r_low : P.dual;
    // advantage 0: nothing, past fp32's range of ratios too (0 * inf)
    const float u = A == 0.0f && r == kInf ? 0.0f : -A * r;
    o.pg = off ? -A * bound : u;
    o.off = off ? 1.0f : 0.0f;
    o.old_kl = exp_beyond_linear(d, r);
    o.grad = off ? 0.0f : u;
    o.kl = 0.0f;
    if (has_ref) {
        const float k = logp - ref;
        float dk;
        if (P.kl == ADAMW_KL_K1) {
            o.kl = k;
            dk = 1.0f;
        } else if (P.kl == ADAMW_KL_K2) {
            o.kl = 0.5f * k * k;
            dk = k;
        } else {
            const float e = expf(-k);
            o.kl = exp_beyond_linear(-k, e);
            // 1 - exp(-k): from the estimate where that is small, not where k
            // would round it away
            dk = fabsf(k) < 0.7f ? k - o.kl : 1.0f - e;
        }
        // without a coefficient the estimate is reported only, and a
        // reference that is -inf somewhere does not reach the gradient
        if (P.kl_coef != 0.0f) o.grad = fmaf(P.kl_coef, dk, o.grad);
    }
    return o;
}

// ---------------------------------------------------------- host helpers --

inline bool launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return true;
    cudaGetLastError();  // not the next caller's error
    adamw::set_cuda_error(what, cudaGetErrorString(e));
    return false;
}

// One launch with programmatic stream serialization, in clusters of `cluster`
// CTAs, with `smem` bytes of dynamic shared memory.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), uint32_t grid, int block, int cluster, size_t smem,
                   cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(unsigned(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kMaxCount = 2147483647;

inline Tokens tokens_of(const adamw_tokens_t* t, const int64_t* targets, int64_t ignore) {
    Tokens k = {};
    k.n = uint32_t(t->n);
    k.sequences = uint32_t(t->sequences);
    k.length = t->offsets || t->n == 0 ? 1u : uint32_t(t->n / t->sequences);
    k.offsets = t->offsets;
    k.mask = t->mask;
    k.targets = targets;
    k.ignore = ignore;
    return k;
}

inline Policy policy_of(const adamw_policy_t* p) {
    Policy k;
    k.r_low = 1.0f - p->clip_low;
    k.r_high = 1.0f + p->clip_high;
    k.d_low = float(std::log1p(-double(p->clip_low)));
    k.d_high = float(std::log1p(double(p->clip_high)));
    k.dual = p->dual_clip;
    k.d_dual = p->dual_clip > 0.0f ? float(std::log(double(p->dual_clip))) : kInf;
    k.kl_coef = p->kl_coef;
    k.entropy_coef = p->entropy_coef;
    k.inv_divisor = p->reduce == ADAMW_REDUCE_FIXED ? 1.0f / p->divisor : 0.0f;
    k.grad_scale = p->grad_scale;
    k.kl = p->kl;
    k.reduce = p->reduce;
    k.per_token = p->advantage_per_token;
    return k;
}

inline int dtype_size(int32_t dt) {
    return dt == ADAMW_DTYPE_FP32 ? 4 : dt == ADAMW_DTYPE_BF16 || dt == ADAMW_DTYPE_FP16 ? 2 : 0;
}

}  // namespace

namespace adamw {

// Shared by the entry points' files (policy_loss.cu, token_logprob.cu).
int check_tokens(const adamw_tokens_t* t);
int check_policy(const adamw_policy_t* p);
// Counts the tokens of `targets` (or of the tokens' mask, or all) into the
// workspace's Counts, and zeroes its ticket.
int launch_counts(const adamw_tokens_t* t, const int64_t* targets, int64_t ignore, void* workspace,
                  cudaStream_t st);
// counted: launch_counts has run on this workspace, and nothing since.
int launch_policy(const adamw_tokens_t* t, const adamw_policy_t* p, const int64_t* targets,
                  int64_t ignore, bool counted, const float* logp, const float* old_logp,
                  const float* ref_logp, const float* advantages, const float* entropy, float* stats, int64_t* counts,
                  float* d_logp, float* d_entropy, void* workspace, cudaStream_t st);

}  // namespace adamw
