// orthogonalize.cu -- Newton-Schulz orthogonalisation of lists of matrices, and
// the Muon step around it.
//
// A call is: the norms of the matrices, their scaled copies in fp16, and three
// products a step,
//     gram   G = X X^T             (symmetric: the tiles on and below the diagonal)
//     poly   Q = b G + c G G       (likewise)
//     apply  X <- a X + Q X
// all matrices of a list in one launch each.  A matrix with more rows than
// columns takes X^T X and X Q: its operands are then read along the other
// dimension, and nothing is transposed.
//
// Numbers.  Everything between the products is fp16 at 2^12 times its value:
// X's singular values stay below 1.3, so |X| and |G| are below 2, |Q| below 4
// with the usual coefficients (16 would overflow), and the small entries of
// large matrices (2^-12 of the norm in a 4096 x 4096 one) stay normal numbers.
// fp16's 11 bits carry an eighth of bf16's rounding errors: bf16 was 1e-2 (random
// matrices) to 2e-1 (rank 64 of 768) off the exact iteration, this is 5e-4 to
// 2.5e-3 above a side of 32 (3.3e-3 the worst of 205000).  X is kept as hi + lo, two fp16: each step multiplies an error of X in
// a direction without singular value by a = 3.44, and a rounding of X itself
// would be such an error; the rounding of the products' operands (hi alone) is
// multiplied by Q, which vanishes in such directions.  lo is as fine as fp16's
// subnormals: 2^-24 beside entries of 2^12 X.
// Thin matrices (a side of at most 128) have few singular values, whose errors do
// not average out: their Q is kept as two fp16 as well, and Q X is three products
// (a small sample of sides of 1 to 4: up to 6.7e-3 off without, 3.5e-3 with).  Up to a
// side of 32 (kFineSide) G is formed from both fp16 of X and kept as two as well;
// in one it left up to 8.9e-3 (the worst of 16800 random matrices of a side of 2;
// 5, 5.4e-3; 8, 3.3e-3; 32, 2.1e-3), in two 8.5e-5.  It costs 8 x 128 19 -> 26 us, 32 x
// 1000 27 -> 33, and a long Gram product thrice its steps (16 x 8192 243 -> 615), so
// sides above, whose worst is below bf16's half step (2^-8), keep one.
#include <algorithm>
#include <atomic>
#include <exception>
#include <new>
#include <vector>

#include "adamw_matrix.h"
#include "tensor_product.cuh"

namespace {

constexpr float kScale = 4096.0f, kUnscale = 1.0f / 4096.0f;

using Fp16 = Elem<ADAMW_DTYPE_FP16>;

// Matrices of one shape, whose working copies lie one after the other.
struct Shape {
    int64_t stride, small_stride;   // elements between matrices (of X, of G)
    int32_t rows, cols, ld;         // ld: cols up to a multiple of 16
    int32_t side, small_ld;         // of G
    bool thin;                      // Q is kept as two fp16
    bool fine;                      // and G, from both of X's
    int32_t count, first;           // matrices, and the first one's number in the list
};

constexpr int kMaxShapes = 8;   // in a launch
constexpr int kFineSide = 32;   // up to which G is two fp16, from both of X's

// ------------------------------------------------------- norms and copies --

// Where a plan's matrices are.
struct MuonMatrix {
    uint16_t* param;
    const uint16_t* grad;
    void* momentum;
    float* master;
};

// The matrices of a call without a plan.
struct Batch {
    char* data;
    int64_t batch_stride, row_stride;
    int32_t dtype;
    int32_t vector;   // kAnyRows, ...
};

constexpr int kNormThreads = 256;
constexpr int kBatch = 4;   // vectors of eight elements in flight in a thread
constexpr int kLeastPiece = kNormThreads * kBatch;

// Vectors that a CTA takes of a list of this many: four batches, one where the
// list would give the GPU fewer than two CTAs an SM (norm and copy of three 515 x
// 1031 fp32: 25 us with four, 19 with one).
inline int32_t piece_size(int64_t vecs) { return vecs / (4 * kLeastPiece) >= 304 ? 4 * kLeastPiece : kLeastPiece; }

struct CopyShape {
    Shape s;
    uint16_t *hi, *lo;
    int32_t pieces;        // of a matrix
    int32_t first_piece;   // of the shape, in the launch
    int32_t first_sum;     // of the shape, in the list
};

template <bool MUON>
struct CopyParams {
    CopyShape shapes[kMaxShapes];
    int32_t n;
    int32_t piece;     // vectors of one
    double* sums;      // by piece
    float eps;
    // without a plan
    Batch src;
    // a plan's
    const MuonMatrix* table;
    const adamw_muon_hparams_t* hp;
    int32_t* nonfinite;
    int32_t nesterov;
};

__device__ __forceinline__ void store8_any(char* data, int64_t at, int32_t dtype, bool vector, int n, const float (&v)[8]) {
    if (dtype == ADAMW_DTYPE_FP32) {
        using E = Elem<ADAMW_DTYPE_FP32>;
        if (vector && n >= 8) {
            *reinterpret_cast<uint4*>(data + at * 4) = E::pack(v);
            *reinterpret_cast<uint4*>(data + at * 4 + 16) = E::pack(v + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) E::store(data, at + i, v[i]);
        }
    } else if (dtype == ADAMW_DTYPE_BF16) {
        using E = Elem<ADAMW_DTYPE_BF16>;
        if (vector && n >= 8) *reinterpret_cast<uint4*>(data + at * 2) = E::pack(v);
        else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) E::store(data, at + i, v[i]);
        }
    } else {
        if (vector && n >= 8) *reinterpret_cast<uint4*>(data + at * 2) = Fp16::pack(v);
        else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) Fp16::store(data, at + i, v[i]);
        }
    }
}

// What eight elements are read as, so that several vectors' loads are in flight
// before the first is looked at: the source (DT), or the gradient in c and the
// momentum (DT) in a and b.
struct Raw {
    uint4 a, b, c;
};

template <int DT>
__device__ __forceinline__ void load_raw(const char* data, int64_t at, bool vector, int n, uint4* a, uint4* b) {
    using E = Elem<DT>;
    const char* p = data + at * E::kSize;
    if (vector) {
        *a = *reinterpret_cast<const uint4*>(p);
        if (E::kSize == 4) *b = *reinterpret_cast<const uint4*>(p + 16);
        return;
    }
    if (E::kSize == 4) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0;
        *a = make_uint4(w[0], w[1], w[2], w[3]);
        *b = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0;
        *a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}
template <int DT>
__device__ __forceinline__ void unpack_raw(uint4 a, uint4 b, float (&v)[8]) {
    Elem<DT>::unpack(a, v);
    if (Elem<DT>::kSize == 4) Elem<DT>::unpack(b, v + 4);
}

// Eight elements of what is orthogonalised: the source, or the step's update
// of gradient and momentum (then the new momentum in `m`).
template <bool MUON, int DT>
struct Source {
    const char *data, *grad;
    int64_t ld;
    int32_t cols;
    float mu;
    bool vector, nesterov;
    __device__ Source(const CopyParams<MUON>& p, const CopyShape& c, int matrix) {
        cols = c.s.cols;
        if (MUON) {
            const MuonMatrix t = p.table[c.s.first + matrix];
            data = static_cast<const char*>(t.momentum);
            grad = reinterpret_cast<const char*>(t.grad);
            ld = cols;
            mu = p.hp->momentum;
            nesterov = p.nesterov != 0;
            vector = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(data) | reinterpret_cast<uintptr_t>(grad)) % 16 == 0;
        } else {
            data = p.src.data + matrix * p.src.batch_stride * Elem<DT>::kSize;
            ld = p.src.row_stride;
            vector = p.src.vector != 0;
        }
    }
    // a row's last vector may be a part of one
    __device__ __forceinline__ Raw load(int row, int col) const {
        Raw r;
        const int64_t at = row * ld + col;
        const int n = cols - col;   // none of the last one of a row whose copy is wider
        const bool whole = vector && n >= 8;
        load_raw<DT>(data, at, whole, n, &r.a, &r.b);
        if (MUON) load_raw<ADAMW_DTYPE_BF16>(grad, at, whole, n, &r.c, &r.c);
        return r;
    }
    __device__ __forceinline__ void value(const Raw& r, float (&u)[8], float (&m)[8]) const {
        if (MUON) {
            unpack_raw<DT>(r.a, r.b, m);
            unpack_raw<ADAMW_DTYPE_BF16>(r.c, r.c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = fmaf(1.0f - mu, u[i] - m[i], m[i]);
                u[i] = nesterov ? fmaf(mu, m[i] - u[i], u[i]) : m[i];
            }
        } else {
            unpack_raw<DT>(r.a, r.b, u);
        }
    }
    // one element
    __device__ __forceinline__ float one(int row, int col, float* m) const {
        const int64_t at = row * ld + col;
        float u = Elem<DT>::load(data, at);
        if (MUON) {
            const float g = Elem<ADAMW_DTYPE_BF16>::load(grad, at);
            *m = fmaf(1.0f - mu, g - u, u);
            u = nesterov ? fmaf(mu, *m - g, g) : *m;
        }
        return u;
    }
    __device__ __forceinline__ void put_one(int row, int col, float m) const {
        if (MUON) Elem<DT>::store(const_cast<char*>(data), row * ld + col, m);
    }
    __device__ __forceinline__ void put(int row, int col, const float (&m)[8]) const {
        if (MUON) store8_any(const_cast<char*>(data), row * ld + col, DT, vector, cols - col, m);
    }
};

// The shape and the matrix of piece i, which becomes its number in the matrix.
template <bool MUON>
__device__ __forceinline__ const CopyShape& piece_of(const CopyParams<MUON>& p, int32_t* i, int32_t* matrix) {
    int k = 0;
    while (k + 1 < p.n && p.shapes[k + 1].first_piece <= *i) ++k;
    const CopyShape& c = p.shapes[k];
    *i -= c.first_piece;
    *matrix = *i / c.pieces;
    *i -= *matrix * c.pieces;
    return c;
}

// Where the vectors of piece i lie: rows of ld / 8 vectors, one after the other.
struct Walk {
    uint32_t per, first_col, n;
    int32_t first_row;
    __device__ Walk(const Shape& s, int32_t i, int32_t piece) {
        per = uint32_t(s.ld) / 8;
        const int64_t first = int64_t(i) * piece, left = int64_t(s.rows) * per - first;
        first_row = int32_t(first / per);
        first_col = uint32_t(first - int64_t(first_row) * per);
        n = uint32_t(left < piece ? left : piece);
    }
    __device__ __forceinline__ bool at(int k, int32_t* row, int32_t* col) const {
        const uint32_t v = first_col + uint32_t(k), r = v / per;
        *row = first_row + int32_t(r);
        *col = int32_t(v - r * per) * 8;
        return uint32_t(k) < n;
    }
};

// Sum of squares of each piece.  Eight squares are summed in fp32 and added
// error-free; squares that leave fp32's comfortable range are taken in fp64.
template <bool MUON, int DT>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ CopyParams<MUON> p) {
    __shared__ double part[kNormThreads / 32];
    int32_t i = int32_t(blockIdx.x), matrix;
    const CopyShape& c = piece_of(p, &i, &matrix);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Source<MUON, DT> src(p, c, matrix);
    const Walk walk(c.s, i, p.piece);
    Sum2 total = {0.0f, 0.0f};
    double sum = 0.0;
#pragma unroll 1
    for (int k = 0; k < p.piece / kNormThreads; k += kBatch) {
        Raw raw[kBatch];
        bool in[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            int32_t row, col;
            in[b] = walk.at((k + b) * kNormThreads + int(threadIdx.x), &row, &col);
            if (in[b]) raw[b] = src.load(row, col);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (!in[b]) continue;
            float u[8], m[8];
            src.value(raw[b], u, m);
            float s = 0.0f, any = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(u[e], u[e], s);
            if (s >= 0x1p-100f && s <= 0x1p100f) {
                total.add(s);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) any = any == 0.0f ? u[e] : any;
            if (any == 0.0f) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += double(u[e]) * double(u[e]);
        }
    }
    sum += double(total.hi) + double(total.lo);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int k = 0; k < kNormThreads / 32; ++k) s += part[k];
        p.sums[c.first_sum + matrix * c.pieces + i] = s;
        if (MUON && !(s <= 1.7976931348623157e308)) atomicOr(p.nonfinite, 1);
    }
}

// What brings a matrix of this sum of squares to 2^12 times the norm 1; NaN for
// a sum that is not finite: the matrix has no direction.  Norms of fp32 numbers
// (1e-45 to 4e44) and eps ask for factors beyond fp32: those come in two, of which
// the first, a power of two, keeps every element in range.
struct Scale {
    float by, again;
    template <int N>
    __device__ __forceinline__ void operator()(float (&x)[N]) const {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] *= by;
        if (again == 1.0f) return;
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] *= again;
    }
};
__device__ __forceinline__ Scale scale_of(double sum, float eps) {
    if (!(sum <= 1.7976931348623157e308)) return {sqrtf(-1.0f), 1.0f};
    const double norm = sqrt(sum), s = double(kScale) / (norm > eps ? norm : double(eps));
    const float f = float(s);   // compared as fp32: fp64 arithmetic is slow
    if (f >= 0x1p-100f && f <= 0x1p100f) return {f, 1.0f};
    if (f > 1.0f) return {0x1p100f, float(s * 0x1p-100)};
    return {0x1p-100f, float(s * 0x1p100)};
}

// x at 2^12 times its value, as two fp16.
__device__ __forceinline__ void split8(const float (&x)[8], uint4* hi, uint4* lo) {
    *hi = Fp16::pack(x);
    float h[8], l[8];
    Fp16::unpack(*hi, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) l[e] = x[e] - h[e];
    *lo = Fp16::pack(l);
}

// The scaled copies; a plan's new momentum.
template <bool MUON, int DT>
__global__ void __launch_bounds__(kNormThreads) copy_kernel(const __grid_constant__ CopyParams<MUON> p) {
    __shared__ double part[kNormThreads / 32];
    int32_t i = int32_t(blockIdx.x), matrix;
    const CopyShape& c = piece_of(p, &i, &matrix);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool skip = MUON && *p.nonfinite != 0;
    // the matrix's norm, by every CTA
    double sum = 0.0;
    for (int k = int(threadIdx.x); k < c.pieces; k += kNormThreads) sum += p.sums[c.first_sum + matrix * c.pieces + k];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.0;
    for (int k = 0; k < kNormThreads / 32; ++k) sum += part[k];
    const Scale scale = scale_of(sum, p.eps);
    const Source<MUON, DT> src(p, c, matrix);
    const Walk walk(c.s, i, p.piece);
    uint4* hi = reinterpret_cast<uint4*>(c.hi + matrix * c.s.stride) + int64_t(i) * p.piece;
    uint4* lo = reinterpret_cast<uint4*>(c.lo + matrix * c.s.stride) + int64_t(i) * p.piece;
#pragma unroll 1
    for (int k = 0; k < p.piece / kNormThreads; k += kBatch) {
        Raw raw[kBatch];
        int32_t row[kBatch], col[kBatch];
        bool in[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            in[b] = walk.at((k + b) * kNormThreads + int(threadIdx.x), &row[b], &col[b]);
            if (in[b]) raw[b] = src.load(row[b], col[b]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (!in[b]) continue;
            float u[8], m[8];
            src.value(raw[b], u, m);
            if (MUON && !skip) src.put(row[b], col[b], m);
            scale(u);
            uint4 h, l;
            split8(u, &h, &l);
            const int at = (k + b) * kNormThreads + int(threadIdx.x);   // the copy's rows are whole vectors
            hi[at] = h;
            lo[at] = l;
        }
    }
}

// By the type of the source, or of the momentum.
template <bool MUON>
using CopyKernel = void (*)(CopyParams<MUON>);
template <bool MUON>
CopyKernel<MUON> norm_of(int32_t dtype) {
    return dtype == ADAMW_DTYPE_FP32 ? norm_kernel<MUON, ADAMW_DTYPE_FP32>
           : dtype == ADAMW_DTYPE_BF16 ? norm_kernel<MUON, ADAMW_DTYPE_BF16> : norm_kernel<MUON, MUON ? ADAMW_DTYPE_BF16 : ADAMW_DTYPE_FP16>;
}
template <bool MUON>
CopyKernel<MUON> copy_of(int32_t dtype) {
    return dtype == ADAMW_DTYPE_FP32 ? copy_kernel<MUON, ADAMW_DTYPE_FP32>
           : dtype == ADAMW_DTYPE_BF16 ? copy_kernel<MUON, ADAMW_DTYPE_BF16> : copy_kernel<MUON, MUON ? ADAMW_DTYPE_BF16 : ADAMW_DTYPE_FP16>;
}

// ---------------------------------------------------------------- products --

enum Kind { kGram, kPoly, kApply, kResult, kUpdate };

struct ProductShape {
    CUtensorMap a, b, a_low, b_low;
    // blocks of the epilogue, 32 rows of 64: what it reads (X or G), second fp16 (X's
    // that it reads and writes, Q's that it writes), what it writes, and the
    // mirrored result, 64 rows of 32
    CUtensorMap in, low, result, turned;
    Shape s;
    int32_t m, n, k;                   // the product's own
    int32_t tiles_m, tiles_n, per;     // tiles of a matrix
    int32_t first_tile;
    bool a_mn, b_mn;
    float rate;                        // of the update
};

struct ProductParams {
    ProductShape shapes[kMaxShapes];
    int32_t n, tiles;
    float a, b, c;
    Batch dst;
    const MuonMatrix* table;
    const adamw_muon_hparams_t* hp;
    int32_t* nonfinite;   // a step's: a wait that runs out also keeps it from writing what comes after
    int32_t pretend;      // report as if one had run out
};

__device__ __forceinline__ void gave_up_on(int32_t* nonfinite) {
    if (nonfinite) atomicOr(nonfinite, 2);
}

// LOW_IN, LOW_OUT: X has its second fp16, the next X gets one.  Of G and Q, LOW_IN:
// there are fine shapes (a flag at run time alone slowed all others by 2 to 5 %).
template <int KIND, class S, bool LOW_IN = false, bool LOW_OUT = false>
struct Product {
    using Params = ProductParams;
    static constexpr bool kTail = false, kParts = KIND >= kApply || LOW_IN;
    static constexpr size_t kTable = 0;
    // Eight warps, each with two staged blocks: X, G and their like come and go
    // by TMA, in rows of 128 bytes.  Sectors by threads made four times the requests,
    // and the epilogue longer than the products of up to 2048 k (apply of 16 x 2048^2
    // with both fp16 of X 192 us, of 32 x 512 x 1024 51 us; staged 185 and 41).
    static constexpr int kWarps = 8;
    static constexpr uint32_t kStaging = 8192;
    static constexpr bool kStaged = true;
    static constexpr uint32_t kRing = S::kStageBytes > 32768 ? 147456 : 163840;
    static constexpr bool kSymmetric = KIND == kGram || KIND == kPoly;
    // tiles of rows to a tile of columns
    static constexpr int kRatio = S::kCols / S::kRows;

    struct Out {
        // by value: read through a pointer to the arguments, each of these cost
        // a trip to L1 in every vector
        int32_t m, n, cols;
        int32_t matrix, row, col;   // of the CTA's part
        int32_t vector;             // of the result's rows
        bool mirrored, skip, thin, fine;
        const ProductShape* maps;
        char *dst, *param;          // the result, or the master and the parameter
        int64_t dst_ld;
        int32_t dst_type;
        float decay, rate, a, b, c;
    };
    __device__ static bool bf16(const Params&) { return false; }
    __device__ static void gave_up(const Params& p) { gave_up_on(p.nonfinite); }
    __device__ static bool pretend(const Params& p) { return p.pretend != 0; }
    __device__ static void prepare(const Params&, unsigned char*) {}
    __device__ static int tiles(const Params& p, const unsigned char*) { return p.tiles; }
    __device__ static const ProductShape& find(const Params& p, int t, int32_t* matrix, int32_t* m, int32_t* n) {
        int k = 0;
        while (k + 1 < p.n && p.shapes[k + 1].first_tile <= t) ++k;
        const ProductShape& c = p.shapes[k];
        t -= c.first_tile;
        *matrix = t / c.per;
        t -= *matrix * c.per;
        if (kSymmetric) {
            // the lower triangle, its diagonal in squares of kCols: the kRatio
            // rows of square r have r + 1 tiles each
            int32_t r = int32_t((sqrtf(8.0f / kRatio * float(t) + 1.0f) - 1.0f) * 0.5f);
            while (kRatio * r * (r + 1) / 2 > t) --r;
            while (kRatio * (r + 1) * (r + 2) / 2 <= t) ++r;
            t -= kRatio * r * (r + 1) / 2;
            *m = r * kRatio + t / (r + 1);
            *n = t % (r + 1);
        } else {
            // bands of eight tiles of rows, for reuse in L2
            const int32_t band = t / (8 * c.tiles_n), left = c.tiles_m - band * 8, h = left < 8 ? left : 8;
            t -= band * 8 * c.tiles_n;
            *m = band * 8 + t % h;
            *n = t / h;
        }
        return c;
    }
    __device__ static void loads(const Params& p, const unsigned char*, int t, TileLoads& w) {
        int32_t m, n;
        const ProductShape& c = find(p, t, &w.a_z, &m, &n);
        w.b_z = w.a_z;
        w.a = &c.a;
        w.b = &c.b;
        w.a_at = m * S::kRows;
        w.b_at = n * S::kCols;
        w.k_at = 0;
        w.k_len = c.k;
        w.a_mn = c.a_mn;
        w.b_mn = c.b_mn;
        w.part = 0;
        if (kParts && (KIND >= kApply ? c.s.thin : c.s.fine)) {
            w.a_low = &c.a_low;
            w.b_low = &c.b_low;
            w.part = (c.k + kStepK - 1) / kStepK * kStepK;
            w.k_len = 3 * w.part;
        }
    }
    template <class>
    __device__ static Out out(const Params& p, const unsigned char*, int t, uint32_t rank) {
        Out o;
        int32_t m, n;
        const ProductShape& c = find(p, t, &o.matrix, &m, &n);
        o.m = c.m;
        o.n = c.n;
        o.cols = c.s.cols;
        o.row = m * S::kRows + int32_t(rank) * kRowsOfCta;
        o.col = n * S::kCols;
        o.mirrored = kSymmetric && m / kRatio != n;
        o.skip = false;
        o.thin = c.s.thin;
        o.fine = LOW_IN && c.s.fine;
        o.vector = kSectorRows;
        o.a = p.a;
        o.b = p.b;
        o.c = p.c * kUnscale;
        o.maps = &c;
        if constexpr (KIND == kResult) {
            o.dst_type = p.dst.dtype;
            o.dst = p.dst.data + o.matrix * p.dst.batch_stride * (o.dst_type == ADAMW_DTYPE_FP32 ? 4 : 2);
            o.dst_ld = p.dst.row_stride;
            o.vector = p.dst.vector;
        } else if constexpr (KIND == kUpdate) {
            const MuonMatrix t = p.table[c.s.first + o.matrix];
            o.dst = reinterpret_cast<char*>(t.master);
            o.param = reinterpret_cast<char*>(t.param);
            o.dst_ld = c.s.cols;
            const uintptr_t at32 = reinterpret_cast<uintptr_t>(t.master) | reinterpret_cast<uintptr_t>(t.param) | uintptr_t(c.s.cols) * 2;
            o.vector = at32 % 32 == 0 ? kSectorRows : at32 % 16 == 0 ? kHalfRows : kAnyRows;
            o.skip = *p.nonfinite != 0;
            const float lr = p.hp->lr;
            o.decay = 1.0f - lr * p.hp->weight_decay;
            o.rate = lr * c.rate * kUnscale;
        }
        return o;
    }
    __device__ static bool wanted(const Params&, const Out& o, int row, int col) {
        return !o.skip && o.row + row < o.m && o.col + col < o.n;
    }
    // Is the result two fp16?  A thin G or Q is one tile, nothing of it is mirrored.
    __device__ static bool split(const Out& o) { return LOW_OUT || (KIND == kPoly && o.thin) || (KIND == kGram && LOW_IN && o.fine); }
    // X or G at the warp's block from column `col`, into its buffers.
    __device__ static void begin(const Params& p, const Out& o, Staged& s, int col) {
        if (KIND == kGram || !wanted(p, o, s.row, col)) return;
        if (elected()) {
            const bool two = LOW_IN && (KIND != kPoly || o.fine);
            barrier_expect(s.bar, two ? 8192 : 4096);
            load_box<1>(smem_addr(s.one), &o.maps->in, o.col + col, o.row + s.row, o.matrix, s.bar);
            if (two) load_box<1>(smem_addr(s.two), &o.maps->low, o.col + col, o.row + s.row, o.matrix, s.bar);
        }
        __syncwarp();
    }
    __device__ static bool finish(const Params& p, const Out& o, Staged& s, bool) {
        for (int c = s.col; c < s.end; c += kBlock64) {
            if (!wanted(p, o, s.row, c)) continue;
            uint4 hi[KIND == kGram ? 1 : 8], low[LOW_IN && KIND >= kApply ? 8 : 1];
            if constexpr (KIND != kGram) {
                if (!s.wait.warp(s.bar, s.turn)) return false;
                s.turn ^= 1;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    hi[j] = *unit_of(s.one, s.lane, j);
                    if constexpr (LOW_IN && KIND >= kApply) low[j] = *unit_of(s.two, s.lane, j);
                }
                __syncwarp();
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[32];
                tmem_load(s.acc + uint32_t(c + half * 32), v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float* y = v + j * 8;
                    float h[8];
                    if constexpr (KIND == kGram) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] *= kUnscale;
                    } else if constexpr (KIND == kPoly) {
                        Fp16::unpack(hi[half * 4 + j], h);
                        if (LOW_IN && o.fine) {   // still there: it is overwritten below, unit by unit
                            float l[8];
                            Fp16::unpack(*unit_of(s.two, s.lane, half * 4 + j), l);
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] += l[e];
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = fmaf(o.b, h[e], o.c * y[e]);
                    } else {
                        Fp16::unpack(hi[half * 4 + j], h);
                        if constexpr (LOW_IN) {
                            float l[8];
                            Fp16::unpack(low[half * 4 + j], l);
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] += l[e];
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = fmaf(o.a, h[e], y[e] * kUnscale);
                    }
                    if constexpr (KIND <= kApply) {
                        if (split(o)) {
                            uint4 a, b;
                            split8(*reinterpret_cast<float(*)[8]>(y), &a, &b);
                            *unit_of(s.one, s.lane, half * 4 + j) = a;
                            *unit_of(s.two, s.lane, half * 4 + j) = b;
                        } else {
                            *unit_of(s.one, s.lane, half * 4 + j) = Fp16::pack(y);
                        }
                    }
                }
                if constexpr (kSymmetric) {
                    if (o.mirrored) {   // row e of 64 bytes: the block's column
                        __half* turned = reinterpret_cast<__half*>(s.two) + half * 32 * 32 + s.lane;
#pragma unroll
                        for (int e = 0; e < 32; ++e) turned[e * 32] = __float2half_rn(v[e]);
                    }
                }
                if constexpr (KIND == kResult || KIND == kUpdate) last(p, o, s, c + half * 32, v);
            }
            if constexpr (KIND <= kApply) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (elected()) {
                    store_box(&o.maps->result, o.col + c, o.row + s.row, o.matrix, smem_addr(s.one));
                    if (split(o)) store_box(&o.maps->low, o.col + c, o.row + s.row, o.matrix, smem_addr(s.two));
                    if constexpr (kSymmetric) {
                        if (o.mirrored) store_box(&o.maps->turned, o.row + s.row, o.col + c, o.matrix, smem_addr(s.two));
                    }
                    stores_read();
                }
                __syncwarp();
            }
            if (c + kBlock64 < s.end) begin(p, o, s, c + kBlock64);
        }
        return true;
    }
    // 32 columns of the result, or of the update.
    __device__ static void last(const Params& p, const Out& o, Staged& s, int c, float (&v)[32]) {
        const int row = s.row + s.lane, left = o.cols - o.col - c;
        const int64_t to = int64_t(o.row + row) * o.dst_ld + o.col + c;
        const bool whole = o.vector == kSectorRows;
        if constexpr (KIND == kResult) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= kUnscale;
        }
        if (o.vector) {
            if (o.row + row >= o.m) return;
            if constexpr (KIND == kResult) {
                store_row(o.dst + to * (o.dst_type == ADAMW_DTYPE_FP32 ? 4 : 2), o.dst_type, v, left, whole);
            } else {
                float w[32];
                load_row<ADAMW_DTYPE_FP32>(o.dst + to * 4, w, left, whole);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = fmaf(-o.rate, v[e], o.decay * w[e]);
                store_row<ADAMW_DTYPE_FP32>(o.dst + to * 4, v, left, whole);
                store_row<ADAMW_DTYPE_BF16>(o.param + to * 2, v, left, whole);
            }
            return;
        }
        // rows that are not whole vectors: element by element, neighbours by
        // neighbouring lanes, through the first buffer
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(unit_of(s.one, s.lane, i)) = *reinterpret_cast<float4*>(v + i * 4);
        __syncwarp();
#pragma unroll 4
        for (int r = 0; r < 32; ++r)
            store_one(p, o, s.row + r, c + s.lane, reinterpret_cast<const float*>(unit_of(s.one, r, s.lane / 4))[s.lane % 4]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the next block comes by TMA
        __syncwarp();
    }
    __device__ static void store_one(const Params& p, const Out& o, int row, int col, float v) {
        if (!wanted(p, o, row, col)) return;
        const int64_t to = int64_t(o.row + row) * o.dst_ld + o.col + col;
        if constexpr (KIND == kResult) {
            store_as(o.dst, to, o.dst_type, v);
        } else if constexpr (KIND == kUpdate) {
            float* w = reinterpret_cast<float*>(o.dst) + to;
            v = fmaf(-o.rate, v, o.decay * *w);
            *w = v;
            store_as(o.param, to, ADAMW_DTYPE_BF16, v);
        }
    }
};

// -------------------------------------------------------------------- host --

constexpr int64_t kMaxSide = int64_t(1) << 20;
constexpr int64_t kMaxElems = int64_t(1) << 40, kMaxMatrices = int64_t(1) << 20;

int64_t up(int64_t n, int64_t by) { return (n + by - 1) / by * by; }

Shape shape_of(int64_t rows, int64_t cols) {
    Shape s = {};
    s.rows = int32_t(rows);
    s.cols = int32_t(cols);
    s.ld = int32_t(up(cols, 16));   // whole 32-byte sectors
    s.stride = rows * s.ld;
    s.side = s.rows <= s.cols ? s.rows : s.cols;
    s.small_ld = int32_t(up(s.side, 16));
    s.small_stride = int64_t(s.side) * s.small_ld;
    s.thin = s.side <= 128;
    s.fine = s.side <= kFineSide;
    return s;
}
int64_t vecs_of(const Shape& s) { return int64_t(s.rows) * (s.ld / 8); }
int64_t pieces_of(const Shape& s, int32_t piece) { return (vecs_of(s) + piece - 1) / piece; }

// The working copies of a shape.
struct Buffers {
    uint16_t *x[2], *lo, *gram, *poly;
    uint16_t* poly_lo;   // Q's, and before it G's: a thin matrix's is one tile, which reads all of G first
};
// A shape's buffers at `at`, each at a multiple of 256 bytes; the bytes they take.
int64_t place(const Shape& s, char* at, Buffers* b) {
    const int64_t big = up(s.stride * s.count * 2, 256), small = up(s.small_stride * s.count * 2, 256);
    if (b) {
        b->x[0] = reinterpret_cast<uint16_t*>(at);
        b->x[1] = reinterpret_cast<uint16_t*>(at + big);
        b->lo = reinterpret_cast<uint16_t*>(at + 2 * big);
        b->gram = reinterpret_cast<uint16_t*>(at + 3 * big);
        b->poly = reinterpret_cast<uint16_t*>(at + 3 * big + small);
        b->poly_lo = s.thin ? reinterpret_cast<uint16_t*>(at + 3 * big + 2 * small) : nullptr;
    }
    return 3 * big + (s.thin ? 3 : 2) * small;
}

// The products of one group of shapes: at most kMaxShapes.
struct Group {
    int n = 0;
    Shape shapes[kMaxShapes];
    Buffers buffers[kMaxShapes];
    float rate[kMaxShapes];
};

// Tiles of a matrix.
template <class S>
int64_t tiles_of(const Shape& s, int kind) {
    const int64_t side = s.side;
    if (kind != kGram && kind != kPoly) return (up(s.rows, S::kRows) / S::kRows) * (up(s.cols, S::kCols) / S::kCols);
    const int64_t m = up(side, S::kRows) / S::kRows, n = up(side, S::kCols) / S::kCols, ratio = S::kCols / S::kRows;
    return ratio * n * (n + 1) / 2 - (ratio * n - m) * n;   // the last square may have fewer rows
}

// The products' arguments, but for the coefficients.  which: X's buffer.
template <class S>
bool fill(const Group& g, int kind, int which, ProductParams* p) {
    memset(p, 0, sizeof *p);
    p->n = g.n;
    int64_t tiles = 0;
    for (int i = 0; i < g.n; ++i) {
        const Shape& s = g.shapes[i];
        const Buffers& b = g.buffers[i];
        ProductShape& q = p->shapes[i];
        q.s = s;
        q.rate = g.rate[i];
        const bool wide = s.rows <= s.cols;
        bool ok;
        if (kind == kGram) {
            q.a_mn = q.b_mn = !wide;
            q.m = q.n = s.side;
            q.k = wide ? s.cols : s.rows;
            ok = tensor_map(&q.a, false, b.x[which], s.count, s.rows, s.cols, s.ld, s.stride, wide ? kRowsOfCta : kStepK) &&
                 tensor_map(&q.b, false, b.x[which], s.count, s.rows, s.cols, s.ld, s.stride, wide ? S::kBRows : kStepK);
            ok = ok && tensor_map(&q.result, false, b.gram, s.count, s.side, s.side, s.small_ld, s.small_stride, 32) &&
                 tensor_map(&q.turned, false, b.gram, s.count, s.side, s.side, s.small_ld, s.small_stride, 64, 32);
            if (ok && s.fine)
                ok = tensor_map(&q.a_low, false, b.lo, s.count, s.rows, s.cols, s.ld, s.stride, wide ? kRowsOfCta : kStepK) &&
                     tensor_map(&q.b_low, false, b.lo, s.count, s.rows, s.cols, s.ld, s.stride, wide ? S::kBRows : kStepK) &&
                     tensor_map(&q.low, false, b.poly_lo, s.count, s.side, s.side, s.small_ld, s.small_stride, 32);
        } else if (kind == kPoly) {
            q.m = q.n = q.k = s.side;
            ok = tensor_map(&q.a, false, b.gram, s.count, s.side, s.side, s.small_ld, s.small_stride, kRowsOfCta) &&
                 tensor_map(&q.b, false, b.gram, s.count, s.side, s.side, s.small_ld, s.small_stride, S::kBRows);
            ok = ok && tensor_map(&q.in, false, b.gram, s.count, s.side, s.side, s.small_ld, s.small_stride, 32) &&
                 tensor_map(&q.result, false, b.poly, s.count, s.side, s.side, s.small_ld, s.small_stride, 32) &&
                 tensor_map(&q.turned, false, b.poly, s.count, s.side, s.side, s.small_ld, s.small_stride, 64, 32);
            if (ok && s.thin) ok = tensor_map(&q.low, false, b.poly_lo, s.count, s.side, s.side, s.small_ld, s.small_stride, 32);
            if (ok && s.fine)
                ok = tensor_map(&q.a_low, false, b.poly_lo, s.count, s.side, s.side, s.small_ld, s.small_stride, kRowsOfCta) &&
                     tensor_map(&q.b_low, false, b.poly_lo, s.count, s.side, s.side, s.small_ld, s.small_stride, S::kBRows);
        } else {
            q.m = s.rows;
            q.n = s.cols;
            q.k = s.side;
            q.b_mn = wide;
            ok = tensor_map(wide ? &q.b : &q.a, false, b.x[which], s.count, s.rows, s.cols, s.ld, s.stride, wide ? kStepK : kRowsOfCta) &&
                 tensor_map(wide ? &q.a : &q.b, false, b.poly, s.count, s.side, s.side, s.small_ld, s.small_stride,
                            wide ? kRowsOfCta : S::kBRows);
            if (ok && s.thin)
                ok = tensor_map(wide ? &q.b_low : &q.a_low, false, b.lo, s.count, s.rows, s.cols, s.ld, s.stride, wide ? kStepK : kRowsOfCta) &&
                     tensor_map(wide ? &q.a_low : &q.b_low, false, b.poly_lo, s.count, s.side, s.side, s.small_ld, s.small_stride,
                                wide ? kRowsOfCta : S::kBRows);
            ok = ok && tensor_map(&q.in, false, b.x[which], s.count, s.rows, s.cols, s.ld, s.stride, 32) &&
                 tensor_map(&q.low, false, b.lo, s.count, s.rows, s.cols, s.ld, s.stride, 32) &&
                 tensor_map(&q.result, false, b.x[which ^ 1], s.count, s.rows, s.cols, s.ld, s.stride, 32);
        }
        if (!ok) return false;
        q.tiles_m = int32_t(up(q.m, S::kRows) / S::kRows);
        q.tiles_n = int32_t(up(q.n, S::kCols) / S::kCols);
        const int64_t per = tiles_of<S>(s, kind);
        q.per = int32_t(per);
        q.first_tile = int32_t(tiles);
        tiles += per * s.count;
        if (tiles > kMaxCount) return false;
    }
    p->tiles = int32_t(tiles);
    return true;
}

struct Device {
    int sms = 0, pairs = 0;
};

template <class P, class S>
bool allow() {
    return launched(cudaFuncSetAttribute(tile_kernel<P, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(tile_smem<P>())), "cudaFuncSetAttribute");
}

template <class S>
bool allow_all() {
    return allow<Product<kGram, S>, S>() && allow<Product<kGram, S, true>, S>() && allow<Product<kPoly, S>, S>() &&
           allow<Product<kPoly, S, true>, S>() && allow<Product<kApply, S>, S>() &&
           allow<Product<kApply, S, true>, S>() && allow<Product<kApply, S, true, true>, S>() && allow<Product<kResult, S>, S>() &&
           allow<Product<kResult, S, true>, S>() && allow<Product<kUpdate, S>, S>() && allow<Product<kUpdate, S, true>, S>();
}

// The current device's units; allows the kernels' shared memory there.
bool device_units(Device* d) {
    static thread_local int known = -1;
    static thread_local Device units;
    int device = 0;
    if (!launched(cudaGetDevice(&device), "cudaGetDevice")) return false;
    if (known != device) {
        if (!allow_all<PairTile>() || !allow_all<WideTile>() || !allow_all<SmallTile>()) return false;
        TileUnits u;
        if (!launched(tile_units<Product<kApply, PairTile>>(&u), "tile units")) return false;
        units.sms = u.sms;
        units.pairs = u.pairs;
        known = device;
    }
    *d = units;
    return true;
}

template <class P, class S>
bool launch_product(const ProductParams& p, int units, cudaStream_t st) {
    const uint32_t grid = uint32_t(p.tiles < units ? p.tiles : units) * S::kPair;
    return launched(launch(tile_kernel<P, S>, grid, tile_threads<P>(), S::kPair, tile_smem<P>(), st, p), "product launch");
}
template <class S>
bool launch_kind(int kind, bool fine, bool low_in, bool low_out, const ProductParams& p, int units, cudaStream_t st) {
    switch (kind) {
        case kGram:
            return fine ? launch_product<Product<kGram, S, true>, S>(p, units, st) : launch_product<Product<kGram, S>, S>(p, units, st);
        case kPoly:
            return fine ? launch_product<Product<kPoly, S, true>, S>(p, units, st) : launch_product<Product<kPoly, S>, S>(p, units, st);
        case kApply:
            return !low_in    ? launch_product<Product<kApply, S>, S>(p, units, st)
                   : !low_out ? launch_product<Product<kApply, S, true>, S>(p, units, st)
                              : launch_product<Product<kApply, S, true, true>, S>(p, units, st);
        case kResult:
            return low_in ? launch_product<Product<kResult, S, true>, S>(p, units, st) : launch_product<Product<kResult, S>, S>(p, units, st);
        default:
            return low_in ? launch_product<Product<kUpdate, S, true>, S>(p, units, st) : launch_product<Product<kUpdate, S>, S>(p, units, st);
    }
}

std::atomic<int32_t> g_pretend{0};   // adamw_matrix_test_expire

// The steps of one group, whose copies have been made.  last: kResult or
// kUpdate, with what it needs in `with`.
bool run_steps(const Group& g, const adamw_ortho_t& o, const float* coefs, int last, const ProductParams& with, const Device& d,
               cudaStream_t st) {
    auto row = [&](int k) { return coefs + 3 * (k < o.n_coefficients ? k : o.n_coefficients - 1); };
    bool low_in = true;   // X starts as two fp16
    bool thin = false;    // products of thin matrices take both
    bool fine = false;
    for (int i = 0; i < g.n; ++i) thin = thin || g.shapes[i].thin, fine = fine || g.shapes[i].fine;
    for (int k = 0; k < o.steps; ++k) {
        // by how much the steps after this one multiply an error of X in a
        // direction without singular value; up to 16, X keeps eleven bits.  With both fp16
        // to the end, sides of 129 to 2048 whose rank is an eighth of them are 0.8e-3 off
        // instead of 2.5e-3, but random ones 1.4e-3 to 1.8e-3 instead of 1.1e-3 to 1.5e-3 (G
        // is formed from the first alone, and is then not that of the X it multiplies),
        // and lists are 1.5 to 5 % slower.
        double later = 1.0;
        for (int i = k + 1; i < o.steps; ++i) later *= std::fabs(double(row(i)[0]));
        const bool low_out = low_in && (later > 16.0 || (thin && k + 1 < o.steps));
        const float* c = row(k);
        for (int kind = kGram; kind <= kApply; ++kind) {
            const int which = kind == kApply && k + 1 == o.steps ? last : kind;
            TileChoice choice = {{0, 0, 0}};
            int64_t steps = 0;
            for (int i = 0; i < g.n; ++i) {
                const Shape& s = g.shapes[i];
                choice.tiles[kPairShape] += tiles_of<PairTile>(s, kind) * s.count;
                choice.tiles[kWideShape] += tiles_of<WideTile>(s, kind) * s.count;
                choice.tiles[kSmallShape] += tiles_of<SmallTile>(s, kind) * s.count;
                // the list's average
                steps += up(kind == kGram ? std::max(s.rows, s.cols) : s.side, kStepK) / kStepK * tiles_of<PairTile>(s, kind) * s.count;
            }
            steps /= choice.tiles[kPairShape];
            const int shape = choose_shape(choice, steps, d.pairs, d.sms);
            ProductParams p;
            if (!(shape == kPairShape   ? fill<PairTile>(g, kind, k & 1, &p)
                  : shape == kWideShape ? fill<WideTile>(g, kind, k & 1, &p)
                                        : fill<SmallTile>(g, kind, k & 1, &p)))
                return false;
            p.a = c[0];
            p.b = c[1];
            p.c = c[2];
            p.dst = with.dst;
            p.table = with.table;
            p.hp = with.hp;
            p.nonfinite = with.nonfinite;
            p.pretend = g_pretend;
            if (!(shape == kPairShape   ? launch_kind<PairTile>(which, fine, low_in, low_out, p, d.pairs, st)
                  : shape == kWideShape ? launch_kind<WideTile>(which, fine, low_in, low_out, p, d.sms, st)
                                        : launch_kind<SmallTile>(which, fine, low_in, low_out, p, d.sms, st)))
                return false;
        }
        low_in = low_out;
    }
    return true;
}

int check_ortho(const adamw_ortho_t* o) {
    if (!o || o->steps < 1 || o->steps > 32 || o->n_coefficients < 1 || o->n_coefficients > 32 || !o->coefficients ||
        !(o->eps > 0.0f) || !std::isfinite(o->eps))
        return ADAMW_ERR_INVALID_ARG;
    for (int i = 0; i < 3 * o->n_coefficients; ++i)
        if (!std::isfinite(o->coefficients[i])) return ADAMW_ERR_INVALID_ARG;
    return ADAMW_OK;
}

bool sizes_fit(int64_t batch, int64_t rows, int64_t cols) {
    return batch >= 0 && rows >= 0 && cols >= 0 && rows <= kMaxSide && cols <= kMaxSide && batch <= kMaxMatrices &&
           (rows == 0 || cols == 0 || batch <= kMaxElems / (rows * cols));
}

int check_matrices(const adamw_matrices_t* m, bool written) {
    if (!m || m->batch < 0 || m->rows < 0 || m->cols < 0 || m->batch_stride < 0 || m->row_stride < 0 || dtype_size(m->dtype) == 0)
        return ADAMW_ERR_INVALID_ARG;
    if (!sizes_fit(m->batch, m->rows, m->cols) || m->row_stride > (int64_t(1) << 40) || m->batch_stride > (int64_t(1) << 40))
        return ADAMW_ERR_TOO_LARGE;
    if (m->batch * m->rows * m->cols == 0) return ADAMW_OK;
    if (!m->data) return ADAMW_ERR_INVALID_ARG;
    if (written && !apart(*m)) return ADAMW_ERR_INVALID_ARG;
    return aligned(m->data, uintptr_t(dtype_size(m->dtype))) ? ADAMW_OK : ADAMW_ERR_MISALIGNED;
}

Batch batch_of(const adamw_matrices_t& m) {
    return {static_cast<char*>(m.data), m.batch_stride, m.row_stride, m.dtype, rows_at(m)};
}

// Pieces of the shapes of a launch, from the list's sum number `sum` on.
template <bool MUON>
int64_t fill_copies(const Group& g, const int32_t* first_sum, int32_t piece, CopyParams<MUON>* p) {
    int64_t pieces = 0;
    p->n = g.n;
    p->piece = piece;
    for (int i = 0; i < g.n; ++i) {
        CopyShape& c = p->shapes[i];
        c.s = g.shapes[i];
        c.hi = g.buffers[i].x[0];
        c.lo = g.buffers[i].lo;
        c.pieces = int32_t(pieces_of(c.s, piece));
        c.first_piece = int32_t(pieces);
        c.first_sum = first_sum[i];
        pieces += int64_t(c.pieces) * c.s.count;
    }
    return pieces;
}

}  // namespace

#include "orthogonalize_small.cuh"

namespace adamw {
int ortho_status(int32_t* out) {
    int32_t v = 0;
    const int32_t zero = 0;
    if (!launched(cudaMemcpyFromSymbol(&v, g_tile_status, 4), "cudaMemcpyFromSymbol") ||
        !launched(cudaMemcpyToSymbol(g_tile_status, &zero, 4), "cudaMemcpyToSymbol"))
        return ADAMW_ERR_CUDA;
    *out |= v;
    return ADAMW_OK;
}
int expert_status(int32_t* out);
}  // namespace adamw

extern "C" int adamw_matrix_status(int32_t* out) {
    if (!out) return ADAMW_ERR_INVALID_ARG;
    *out = 0;
    if (!launched(cudaDeviceSynchronize(), "cudaDeviceSynchronize")) return ADAMW_ERR_CUDA;
    const int rc = adamw::ortho_status(out);
    return rc != ADAMW_OK ? rc : adamw::expert_status(out);
}

extern "C" void adamw_matrix_test_expire(int32_t on) { g_pretend = on != 0; }

extern "C" int64_t adamw_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols) {
    if (!sizes_fit(batch, rows, cols) || batch * rows * cols == 0) return 0;
    Shape s = shape_of(rows, cols);
    s.count = int32_t(batch);
    return up(pieces_of(s, piece_size(vecs_of(s) * batch)) * batch * int64_t(sizeof(double)), 256) + place(s, nullptr, nullptr);
}

extern "C" int adamw_orthogonalize(const adamw_matrices_t* src, const adamw_matrices_t* dst, const adamw_ortho_t* ortho,
                                   void* workspace, adamw_stream_t stream) {
    int rc;
    if ((rc = check_ortho(ortho)) != ADAMW_OK || (rc = check_matrices(src, false)) != ADAMW_OK ||
        (rc = check_matrices(dst, true)) != ADAMW_OK)
        return rc;
    if (src->batch != dst->batch || src->rows != dst->rows || src->cols != dst->cols) return ADAMW_ERR_INVALID_ARG;
    // in place: element for element
    if (overlap(*src, *dst) &&
        (src->data != dst->data || src->dtype != dst->dtype || (src->rows > 1 && src->row_stride != dst->row_stride) ||
         (src->batch > 1 && src->batch_stride != dst->batch_stride)))
        return ADAMW_ERR_INVALID_ARG;
    if (src->batch * src->rows * src->cols == 0) return ADAMW_OK;
    if (!workspace) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return ADAMW_ERR_MISALIGNED;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Device d;
    if (!device_units(&d)) return ADAMW_ERR_CUDA;
    Group g;
    g.n = 1;
    Shape& s = g.shapes[0];
    s = shape_of(src->rows, src->cols);
    s.count = int32_t(src->batch);
    const int32_t piece = piece_size(vecs_of(s) * s.count);
    const int64_t pieces = pieces_of(s, piece) * s.count;
    if (pieces > kMaxCount) return ADAMW_ERR_TOO_LARGE;
    place(s, static_cast<char*>(workspace) + up(pieces * int64_t(sizeof(double)), 256), &g.buffers[0]);
    CopyParams<false> c;
    memset(&c, 0, sizeof c);
    const int32_t first_sum = 0;
    c.sums = static_cast<double*>(workspace);
    c.eps = ortho->eps;
    c.src = batch_of(*src);
    if (small_ctas(s) > 0) {
        SmallParams<false> p;
        memset(&p, 0, sizeof p);
        p.in = c;
        p.dst = batch_of(*dst);
        return launch_small(g, &first_sum, *ortho, ortho->coefficients, src->dtype, d.sms, piece, &p, st) ? ADAMW_OK : ADAMW_ERR_CUDA;
    }
    fill_copies(g, &first_sum, piece, &c);
    if (!launched(launch(norm_of<false>(src->dtype), uint32_t(pieces), kNormThreads, 1, 0, st, c), "norm launch") ||
        !launched(launch(copy_of<false>(src->dtype), uint32_t(pieces), kNormThreads, 1, 0, st, c), "copy launch"))
        return ADAMW_ERR_CUDA;
    ProductParams with;
    memset(&with, 0, sizeof with);
    with.dst = batch_of(*dst);
    return run_steps(g, *ortho, ortho->coefficients, kResult, with, d, st) ? ADAMW_OK : ADAMW_ERR_CUDA;
}

// -------------------------------------------------------------- Muon plan --

struct adamw_muon_plan {
    int device = 0;
    adamw_ortho_t ortho = {};
    std::vector<float> coefs;
    int32_t nesterov = 0, momentum_bf16 = 0, piece = 0;
    std::vector<Group> rounds;                 // one after the other, in the same workspace
    std::vector<std::vector<int32_t>> sums;    // each shape's first sum, by round
    void* block = nullptr;                     // table, sums, workspace
    MuonMatrix* table = nullptr;
    double* d_sums = nullptr;
    char* work = nullptr;
};

namespace {

// Workspace of a round: large enough that a round's products fill the GPU many
// times over, small enough beside a model.
constexpr int64_t kRoundBytes = int64_t(2) << 30;

// Makes a device current for the scope, restoring the caller's.
struct Current {
    int prev = -1;
    bool ok = true;
    explicit Current(int device) {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != device) ok = cudaSetDevice(device) == cudaSuccess; else prev = -1;
    }
    ~Current() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

int check_muon(const adamw_muon_tensor_t* table, int32_t n, const adamw_muon_options_t* o) {
    if (n < 0 || (n > 0 && !table) || !o) return ADAMW_ERR_INVALID_ARG;
    const int rc = check_ortho(&o->ortho);
    if (rc != ADAMW_OK) return rc;
    if ((o->nesterov != 0 && o->nesterov != 1) || (o->scale != ADAMW_MUON_SPECTRAL && o->scale != ADAMW_MUON_RMS) ||
        (o->momentum_dtype != ADAMW_DTYPE_FP32 && o->momentum_dtype != ADAMW_DTYPE_BF16))
        return ADAMW_ERR_INVALID_ARG;
    int64_t matrices = 0;
    for (int32_t k = 0; k < n; ++k) {
        const adamw_muon_tensor_t& t = table[k];
        if (t.batch < 0 || t.rows < 0 || t.cols < 0) return ADAMW_ERR_INVALID_ARG;
        if (!sizes_fit(t.batch, t.rows, t.cols)) return ADAMW_ERR_TOO_LARGE;
        if (t.batch * t.rows * t.cols == 0) continue;
        if (!t.param || !t.grad || !t.momentum || !t.master) return ADAMW_ERR_INVALID_ARG;
        if (!aligned(t.param, 2) || !aligned(t.grad, 2) || !aligned(t.master, 4) ||
            !aligned(t.momentum, o->momentum_dtype == ADAMW_DTYPE_FP32 ? 4 : 2))
            return ADAMW_ERR_MISALIGNED;
        matrices += t.batch;
        if (matrices > kMaxMatrices) return ADAMW_ERR_TOO_LARGE;
    }
    return ADAMW_OK;
}

// No buffer of the list reaches into another: two CTAs would write one place,
// or read what is being written.
int check_apart(const adamw_muon_tensor_t* table, int32_t n, int momentum_size) {
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;
    for (int32_t k = 0; k < n; ++k) {
        const adamw_muon_tensor_t& t = table[k];
        const int64_t numel = t.batch * t.rows * t.cols;
        if (numel == 0) continue;
        const void* at[] = {t.param, t.grad, t.momentum, t.master};
        const int size[] = {2, 2, momentum_size, 4};
        for (int b = 0; b < 4; ++b) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(at[b]);
            spans.emplace_back(p, p + uintptr_t(numel) * uintptr_t(size[b]));
        }
    }
    std::sort(spans.begin(), spans.end());
    for (size_t k = 1; k < spans.size(); ++k)
        if (spans[k].first < spans[k - 1].second) return ADAMW_ERR_INVALID_ARG;
    return ADAMW_OK;
}

int check_device(const void* p, int device, int pageable) {
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        adamw::set_cuda_error("cudaPointerGetAttributes", cudaGetErrorString(cudaGetLastError()));
        return ADAMW_ERR_NOT_ACCESSIBLE;
    }
    const bool ok = a.type == cudaMemoryTypeDevice ? a.device == device
                    : a.type == cudaMemoryTypeManaged ? true
                    : a.type == cudaMemoryTypeHost    ? a.devicePointer == p
                                                      : pageable != 0;
    return ok ? ADAMW_OK : ADAMW_ERR_NOT_ACCESSIBLE;
}

float rate_of(int32_t scale, int64_t rows, int64_t cols) {
    const double r = double(rows), c = double(cols);
    return float(scale == ADAMW_MUON_RMS ? 0.2 * std::sqrt(std::max(r, c)) : std::sqrt(std::max(1.0, r / c)));
}

int create(const adamw_muon_tensor_t* table, int32_t n, const adamw_muon_options_t* o, adamw_muon_plan* P) {
    if (!launched(cudaGetDevice(&P->device), "cudaGetDevice")) return ADAMW_ERR_CUDA;
    int pageable = 0;
    if (!launched(cudaDeviceGetAttribute(&pageable, cudaDevAttrPageableMemoryAccess, P->device), "cudaDeviceGetAttribute"))
        return ADAMW_ERR_CUDA;
    Device d;
    if (!device_units(&d)) return ADAMW_ERR_CUDA;
    P->ortho = o->ortho;
    P->coefs.assign(o->ortho.coefficients, o->ortho.coefficients + 3 * o->ortho.n_coefficients);
    P->ortho.coefficients = nullptr;
    P->nesterov = o->nesterov;
    P->momentum_bf16 = o->momentum_dtype == ADAMW_DTYPE_BF16;
    const int size = P->momentum_bf16 ? 2 : 4;
    // the list's matrices, those of one shape together
    struct Entry {
        int64_t rows, cols;
        int32_t tensor;
    };
    std::vector<Entry> order;
    for (int32_t k = 0; k < n; ++k) {
        const adamw_muon_tensor_t& t = table[k];
        if (t.batch * t.rows * t.cols == 0) continue;
        for (const void* p : {static_cast<const void*>(t.param), t.grad, static_cast<const void*>(t.momentum),
                              static_cast<const void*>(t.master)}) {
            const int rc = check_device(p, P->device, pageable);
            if (rc != ADAMW_OK) return rc;
        }
        order.push_back({t.rows, t.cols, k});
    }
    // the thin ones, and the small ones that have a kernel of their own, last
    auto class_of = [](int64_t rows, int64_t cols) {
        const Shape s = shape_of(rows, cols);
        return small_ctas(s) > 0 ? 2 : s.thin ? 1 : 0;
    };
    std::stable_sort(order.begin(), order.end(), [&](const Entry& a, const Entry& b) {
        const int ca = class_of(a.rows, a.cols), cb = class_of(b.rows, b.cols);
        if (ca != cb) return ca < cb;
        return a.rows * a.cols != b.rows * b.cols ? a.rows * a.cols > b.rows * b.cols : a.rows > b.rows;
    });
    std::vector<MuonMatrix> matrices;
    std::vector<Shape> shapes;
    for (const Entry& e : order) {
        const adamw_muon_tensor_t& t = table[e.tensor];
        if (shapes.empty() || shapes.back().rows != t.rows || shapes.back().cols != t.cols) {
            shapes.push_back(shape_of(t.rows, t.cols));
            shapes.back().first = int32_t(matrices.size());
        }
        for (int64_t b = 0; b < t.batch; ++b) {
            const int64_t at = b * t.rows * t.cols;
            matrices.push_back({static_cast<uint16_t*>(t.param) + at, static_cast<const uint16_t*>(t.grad) + at,
                                static_cast<char*>(t.momentum) + at * size, t.master + at});
            ++shapes.back().count;
        }
    }
    int64_t vecs = 0;
    for (const Shape& s : shapes) vecs += vecs_of(s) * s.count;
    P->piece = piece_size(vecs);
    // rounds: as many matrices as the workspace holds, of at most kMaxShapes shapes
    int64_t sums = 0, work = 0, used = 0;
    for (const Shape& s : shapes) {
        for (int32_t done = 0; done < s.count;) {
            Shape part = s;
            part.first = s.first + done;
            part.count = 1;
            const int64_t one = place(part, nullptr, nullptr);
            const int which = class_of(part.rows, part.cols);
            const bool small = which == 2;
            if (P->rounds.empty() || P->rounds.back().n == kMaxShapes || (!small && used > 0 && used + one > kRoundBytes) ||
                class_of(P->rounds.back().shapes[0].rows, P->rounds.back().shapes[0].cols) != which) {
                P->rounds.emplace_back();
                P->sums.emplace_back();
                used = 0;
            }
            const int64_t room = small ? s.count : (kRoundBytes - used) / one;
            part.count = int32_t(std::min<int64_t>(s.count - done, std::max<int64_t>(room, 1)));
            Group& g = P->rounds.back();
            g.shapes[g.n] = part;
            g.rate[g.n] = rate_of(o->scale, part.rows, part.cols);
            ++g.n;
            P->sums.back().push_back(int32_t(sums));
            sums += pieces_of(part, P->piece) * part.count;
            if (sums > kMaxCount) return ADAMW_ERR_TOO_LARGE;
            if (!small) used += place(part, nullptr, nullptr);
            work = std::max(work, used);
            done += part.count;
        }
    }
    if (matrices.empty()) return ADAMW_OK;
    const int64_t table_bytes = up(int64_t(matrices.size() * sizeof(MuonMatrix)), 256), sum_bytes = up(sums * int64_t(sizeof(double)), 256);
    if (!launched(cudaMalloc(&P->block, size_t(table_bytes + sum_bytes + work)), "cudaMalloc")) return ADAMW_ERR_CUDA;
    P->table = static_cast<MuonMatrix*>(P->block);
    P->d_sums = reinterpret_cast<double*>(static_cast<char*>(P->block) + table_bytes);
    P->work = static_cast<char*>(P->block) + table_bytes + sum_bytes;
    for (Group& g : P->rounds) {
        char* at = P->work;
        for (int i = 0; i < g.n && small_ctas(g.shapes[i]) == 0; ++i) at += place(g.shapes[i], at, &g.buffers[i]);
    }
    const bool ok = launched(cudaMemcpy(P->table, matrices.data(), matrices.size() * sizeof(MuonMatrix), cudaMemcpyHostToDevice),
                             "cudaMemcpy(table)") &&
                    launched(cudaStreamSynchronize(nullptr), "cudaStreamSynchronize");
    return ok ? ADAMW_OK : ADAMW_ERR_CUDA;
}

}  // namespace

extern "C" int adamw_muon_plan_create(const adamw_muon_tensor_t* host_table, int32_t n, const adamw_muon_options_t* options,
                                      adamw_muon_plan_t* out) {
    if (!out) return ADAMW_ERR_INVALID_ARG;
    *out = nullptr;
    int rc = check_muon(host_table, n, options);
    if (rc != ADAMW_OK) return rc;
    adamw_muon_plan* P = new (std::nothrow) adamw_muon_plan;
    if (!P) return ADAMW_ERR_TOO_LARGE;
    try {
        rc = check_apart(host_table, n, options->momentum_dtype == ADAMW_DTYPE_FP32 ? 4 : 2);
        if (rc == ADAMW_OK) rc = create(host_table, n, options, P);
    } catch (const std::exception&) {   // the host has no room for a table
        rc = ADAMW_ERR_TOO_LARGE;
    }
    if (rc != ADAMW_OK) {
        if (P->block) cudaFree(P->block);
        delete P;
        return rc;
    }
    *out = P;
    return ADAMW_OK;
}

extern "C" int adamw_muon_step(adamw_muon_plan_t plan, const adamw_muon_hparams_t* hparams, int32_t* nonfinite,
                               adamw_stream_t stream) {
    if (!plan || !hparams || !nonfinite) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(hparams, 16) || !aligned(nonfinite, 4)) return ADAMW_ERR_MISALIGNED;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Current guard(plan->device);
    if (!guard.ok) {
        adamw::set_cuda_error("cudaSetDevice", cudaGetErrorString(cudaGetLastError()));
        return ADAMW_ERR_CUDA;
    }
    Device d;
    if (!device_units(&d)) return ADAMW_ERR_CUDA;
    if (!launched(cudaMemsetAsync(nonfinite, 0, sizeof(int32_t), st), "cudaMemsetAsync")) return ADAMW_ERR_CUDA;
    CopyParams<true> c;
    memset(&c, 0, sizeof c);
    c.sums = plan->d_sums;
    c.eps = plan->ortho.eps;
    c.table = plan->table;
    c.hp = hparams;
    c.nonfinite = nonfinite;
    c.nesterov = plan->nesterov;
    // every norm first: one gradient that is not finite stops the whole step
    for (size_t r = 0; r < plan->rounds.size(); ++r) {
        const int64_t pieces = fill_copies(plan->rounds[r], plan->sums[r].data(), plan->piece, &c);
        if (!launched(launch(norm_of<true>(plan->momentum_bf16 ? ADAMW_DTYPE_BF16 : ADAMW_DTYPE_FP32), uint32_t(pieces), kNormThreads, 1, 0, st, c), "norm launch")) return ADAMW_ERR_CUDA;
    }
    ProductParams with;
    memset(&with, 0, sizeof with);
    with.table = plan->table;
    with.hp = hparams;
    with.nonfinite = nonfinite;
    const int32_t dtype = plan->momentum_bf16 ? ADAMW_DTYPE_BF16 : ADAMW_DTYPE_FP32;
    for (size_t r = 0; r < plan->rounds.size(); ++r) {
        if (small_ctas(plan->rounds[r].shapes[0]) > 0) {
            SmallParams<true> p;
            memset(&p, 0, sizeof p);
            p.in = c;
            if (!launch_small(plan->rounds[r], plan->sums[r].data(), plan->ortho, plan->coefs.data(), dtype, d.sms, plan->piece, &p, st))
                return ADAMW_ERR_CUDA;
            continue;
        }
        const int64_t pieces = fill_copies(plan->rounds[r], plan->sums[r].data(), plan->piece, &c);
        if (!launched(launch(copy_of<true>(plan->momentum_bf16 ? ADAMW_DTYPE_BF16 : ADAMW_DTYPE_FP32), uint32_t(pieces), kNormThreads, 1, 0, st, c), "copy launch")) return ADAMW_ERR_CUDA;
        if (!run_steps(plan->rounds[r], plan->ortho, plan->coefs.data(), kUpdate, with, d, st)) return ADAMW_ERR_CUDA;
    }
    return ADAMW_OK;
}

extern "C" int adamw_muon_plan_destroy(adamw_muon_plan_t plan) {
    if (!plan) return ADAMW_OK;
    Current guard(plan->device);
    bool ok = guard.ok;
    if (plan->block) {
        ok = ok && launched(cudaDeviceSynchronize(), "cudaDeviceSynchronize");
        ok = launched(cudaFree(plan->block), "cudaFree") && ok;
    }
    delete plan;
    return ok ? ADAMW_OK : ADAMW_ERR_CUDA;
}
