// clip_grads.cu -- the global norm of a list of gradients of several types and
// the clip by it.
//
// Bound by HBM: the list is read for the norm and, its coefficient known only
// after the last element, read again to be scaled (a list that fits the
// 129 MB L2 comes from there the second time).  The OPT-1.3b list, 1.3B fp32
// gradients into bf16: 1.89 ms, 7.0 TB/s over its two reads and one write (the
// copy rate measured on this GPU is 6.67); the OPT-125m list 182 us from fp32,
// 114 us from bf16.  Small lists are bound by the two kernels' latency: a
// million elements in 37 tensors of two types take 6.8 us.
#include <algorithm>
#include <exception>
#include <new>
#include <type_traits>
#include <vector>

#include "losses_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Elements of a tile, the piece of a tensor that a CTA takes at a time: 16384,
// 8192 for lists that give fewer than two of those to each SM.  Measured (bf16
// list, us, largest tile / this rule / at least 2048): 1M elements 4.8 / 4.7 /
// 5.4, 4M 6.8 / 6.2 / 7.9, 16M and above the same; a 1.3B list 1904 with tiles
// of 32768, 1910 of 16384, 1936 of 8192.
constexpr int kMaxTile = 16384, kMinTile = 8192;
constexpr int kNormUnroll = 8;   // 16-byte vectors in flight per thread
constexpr int kScaleVecs = 8;    // likewise, when scaling
constexpr int kMaxGrid = 1216;   // CTAs of the norm pass at most: its partials
constexpr int64_t kMaxTiles = int64_t(1) << 26;

struct alignas(16) Tile {
    const char* src;
    char* dst;
    int32_t len;
    int32_t src_type;
    int32_t vector;   // both 16-byte aligned
    int32_t pad_;
};
static_assert(sizeof(Tile) == 32, "tile layout");

// One CTA's part of the norm: the value x 2^exponent.  The exponent is 0 but
// for sums that leave fp32's range.
struct Partial {
    float x, exponent;
};

// The squares of one thread's elements.  Groups of elements are summed in
// fp32 and added to an error-free running sum.  A group whose sum of squares
// leaves fp32's comfortable range (huge, tiny, inf, NaN) is summed again in
// fp64.
struct SquareSum {
    Sum2 sum;
    double rare;
    // false: the group has to be summed by add_rare
    template <typename E, int U>
    __device__ __forceinline__ bool add(const uint4 (&v)[U]) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E::kVec];
            E::unpack(v[u], x);
#pragma unroll
            for (int i = 0; i < E::kVec; ++i) s[i % 4] = fmaf(x[i], x[i], s[i % 4]);
        }
        const float g = (s[0] + s[1]) + (s[2] + s[3]);
        if (g >= 0x1p-100f && g <= 0x1p100f) {
            sum.add(g);
            return true;
        }
        uint32_t any = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) any |= v[u].x | v[u].y | v[u].z | v[u].w;
        return (any & ~E::kSigns) == 0;   // zeros
    }
    __device__ __forceinline__ void add(float x) {
        const float g = x * x;
        if (g >= 0x1p-100f && g <= 0x1p100f) sum.add(g); else add_rare(x);
    }
    // an fp32 value's square neither overflows nor vanishes in fp64
    __device__ __forceinline__ void add_rare(float x) { rare += double(x) * double(x); }
};

// |x| as bits, which order as |x| does, infinity and then NaN above.
struct MaxBits {
    uint32_t bits;
    template <typename E, int U>
    __device__ __forceinline__ bool add(const uint4 (&v)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E::kVec];
            E::unpack(v[u], x);
#pragma unroll
            for (int i = 0; i < E::kVec; ++i) add(x[i]);
        }
        return true;
    }
    __device__ __forceinline__ void add_rare(float) {}
    __device__ __forceinline__ void add(float x) {
        const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
        bits = b > bits ? b : bits;
    }
};

template <int DT, typename Acc>
__device__ __forceinline__ void norm_tile(const Tile& t, Acc& acc) {
    using E = Elem<DT>;
    int done = 0;
    if (t.vector) {
        const int vecs = t.len / E::kVec;
        constexpr int kBatch = kNormUnroll * kThreads;
        const char* src = t.src + threadIdx.x * 16;
        int base = 0;
        // the batch again, from L2, element by element
        auto again = [&] {
#pragma unroll 1
            for (int u = 0; u < kNormUnroll; ++u) {
                if (base + u * kThreads + int(threadIdx.x) >= vecs) break;
                float x[E::kVec];
                E::unpack(load16(src + (base + u * kThreads) * 16), x);
#pragma unroll
                for (int i = 0; i < E::kVec; ++i) acc.add_rare(x[i]);
            }
        };
        for (; base + kBatch <= vecs; base += kBatch) {
            uint4 v[kNormUnroll];
#pragma unroll
            for (int u = 0; u < kNormUnroll; ++u) v[u] = load16(src + (base + u * kThreads) * 16);
            if (!acc.template add<E, kNormUnroll>(v)) again();
        }
        if (base < vecs) {
            uint4 v[kNormUnroll];
#pragma unroll
            for (int u = 0; u < kNormUnroll; ++u)
                v[u] = base + u * kThreads + int(threadIdx.x) < vecs
                           ? load16(src + (base + u * kThreads) * 16) : make_uint4(0, 0, 0, 0);
            if (!acc.template add<E, kNormUnroll>(v)) again();
        }
        done = vecs * E::kVec;
    }
    for (int i = done + threadIdx.x; i < t.len; i += kThreads) acc.add(E::load(t.src, i));
}

// The larger of two magnitudes, NaN above infinity.
__device__ __forceinline__ float larger(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// The CTA's joined value, in every thread: a tree in fp32 (eight roundings of
// a CTA's value; the CTAs' own average out in the total).
template <bool MAX>
__device__ __forceinline__ float cta_join(float v, float* part) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MAX ? larger(v, o) : v + o;
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v = MAX ? larger(v, part[w]) : v + part[w];
    return v;
}

__device__ __forceinline__ Partial cta_value(const MaxBits& a) {
    __shared__ float part[kWarps];
    return {cta_join<true>(__uint_as_float(a.bits), part), 0.0f};
}
__device__ __forceinline__ Partial cta_value(const SquareSum& a) {
    __shared__ float part[kWarps];
    const bool rare = __syncthreads_or(a.rare != 0.0);
    if (!rare) return {cta_join<false>(a.sum.value(), part), 0.0f};
    __shared__ double wide[kThreads];
    wide[threadIdx.x] = double(a.sum.hi) + double(a.sum.lo) + a.rare;
    __syncthreads();
    double v = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kThreads; ++k) v += wide[k];
    if (!isfinite(v)) return {float(v), 0.0f};
    int e;
    const double m = frexp(v, &e);
    return {float(m), float(e)};
}

// The norm's partial values: tiles dealt round-robin to a resident grid.  The
// next kernel may start once every CTA here has passed its wait, so it may
// read what this one reads before its own.
template <bool MAX>
__global__ void __launch_bounds__(kThreads, 4)
grad_norm_kernel(const Tile* tiles, int32_t n, Partial* partial) {
    Tile t = {};
    if (int32_t(blockIdx.x) < n) t = tiles[blockIdx.x];
    dependency_wait();
    dependency_trigger();
    typename std::conditional<MAX, MaxBits, SquareSum>::type acc = {};
    for (int32_t k = blockIdx.x; k < n; k += gridDim.x) {
        if (k != int32_t(blockIdx.x)) t = tiles[k];
        switch (t.src_type) {
            case ADAMW_DTYPE_BF16: norm_tile<ADAMW_DTYPE_BF16>(t, acc); break;
            case ADAMW_DTYPE_FP16: norm_tile<ADAMW_DTYPE_FP16>(t, acc); break;
            default: norm_tile<ADAMW_DTYPE_FP32>(t, acc); break;
        }
    }
    const Partial p = cta_value(acc);
    if (threadIdx.x == 0) partial[blockIdx.x] = p;
}

// What a call's later kernels need of the norm.
struct Clip {
    const Partial* partial;
    int32_t n;
    int32_t max;   // ADAMW_NORM_MAX
    float max_norm;
    adamw_clip_result_t* result;   // NULL: another kernel of the call writes it
};

// Joins the partial values in their order, the same in every CTA, and gives
// the coefficient in two factors, the second a power of two: a coefficient
// below fp32's normal range (a norm above 1e38 times the limit) keeps its
// digits in the first.  {1, 1} when nothing is scaled.
__device__ __forceinline__ float2 clip_coefficient(const Clip& c) {
    __shared__ Sum2 part[kWarps];
    __shared__ float2 coef;
    Sum2 s = {};
    float top = 0.0f;
    bool wide = false;
    for (int32_t k = threadIdx.x; k < c.n; k += kThreads) {
        const Partial p = c.partial[k];
        s.add(p.x);
        top = larger(top, p.x);
        wide |= p.exponent != 0.0f;
    }
    if (c.max) s = {top, 0.0f};
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float h = __shfl_down_sync(0xffffffffu, s.hi, d), l = __shfl_down_sync(0xffffffffu, s.lo, d);
        if (c.max) s.hi = larger(s.hi, h); else s.join(h, l);
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    wide = __syncthreads_or(wide);
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) {
            if (c.max) s.hi = larger(s.hi, part[w].hi); else s.join(part[w].hi, part[w].lo);
        }
        const float v = c.max ? s.hi : s.value();
        adamw_clip_result_t r = {0.0f, 1.0f, 0, 0};
        float2 two = make_float2(1.0f, 1.0f);
        bool done = false;
        if (!wide && (v == 0.0f || (v > 1e-30f && v < 1e30f))) {
            r.norm = c.max ? v : sqrtf(v);
            const float q = c.max_norm / (r.norm + 1e-6f);
            r.coef = two.x = q < 1.0f ? q : 1.0f;
            done = r.coef >= 0x1p-100f;
        }
        if (!done) {  // out of fp32's reach
            double sum = v;
            if (!c.max) {
                sum = 0.0;
                for (int32_t k = 0; k < c.n; ++k)
                    sum += ldexp(double(c.partial[k].x), int(c.partial[k].exponent));
                sum = sqrt(sum);
            }
            const double q = double(c.max_norm) / (sum + 1e-6);
            r.norm = float(sum);
            r.nonfinite = isfinite(sum) ? 0 : 1;
            const bool scaled = isfinite(sum) && q < 1.0;
            r.coef = scaled ? float(q) : 1.0f;
            two = scaled && q < 0x1p-100 ? make_float2(float(q * 0x1p64), 0x1p-64f) : make_float2(r.coef, 1.0f);
        }
        coef = two;
        if (c.result && blockIdx.x == 0) *c.result = r;
    }
    __syncthreads();
    return coef;
}

__global__ void __launch_bounds__(kThreads) clip_result_kernel(Clip clip) {
    dependency_trigger();
    dependency_wait();
    clip_coefficient(clip);
}

// dst = coef * src for the tiles [first, first + n), all of the kernel's pair
// of types.  In reverse: those that the norm pass read last are the likeliest
// to be in L2 still.
// A CTA's first loads go out before it waits for the norm.
template <int SRC, int DST>
__global__ void __launch_bounds__(kThreads, 4)
grad_scale_kernel(const Tile* tiles, int32_t n, Clip clip) {
    using S = Elem<SRC>;
    using D = Elem<DST>;
    // elements per step: whole 16-byte vectors on both sides
    constexpr int K = S::kVec > D::kVec ? S::kVec : D::kVec;
    constexpr int kIn = K / S::kVec, kOut = K / D::kVec;
    constexpr int U = kScaleVecs / kIn;
    dependency_trigger();
    uint4 v[U][kIn];
    auto load = [&](const Tile& t, int base, int steps) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (base + u * kThreads < steps) {
#pragma unroll
                for (int j = 0; j < kIn; ++j) v[u][j] = load16(t.src + ((base + u * kThreads) * kIn + j) * 16);
            }
    };
    int32_t k = n - 1 - int32_t(blockIdx.x);   // the grid is at most n
    Tile t = tiles[k];
    if (t.vector) load(t, threadIdx.x, t.len / K);
    dependency_wait();
    const float2 coef = clip_coefficient(clip);
    for (bool loaded = true;; loaded = false) {
        if (coef.x != 1.0f || t.dst != t.src) {
            int done = 0;
            if (t.vector) {
                const int steps = t.len / K;
                for (int base = threadIdx.x; base < steps; base += U * kThreads) {
                    if (!loaded) load(t, base, steps);
                    loaded = false;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (base + u * kThreads >= steps) break;
                        float x[K];
#pragma unroll
                        for (int j = 0; j < kIn; ++j) S::unpack(v[u][j], x + j * S::kVec);
#pragma unroll
                        for (int j = 0; j < K; ++j) x[j] = x[j] * coef.x * coef.y;
#pragma unroll
                        for (int j = 0; j < kOut; ++j)
                            store16(t.dst + ((base + u * kThreads) * kOut + j) * 16, D::pack(x + j * D::kVec));
                    }
                }
                done = steps * K;
            }
            for (int i = done + threadIdx.x; i < t.len; i += kThreads)
                D::store(t.dst, i, S::load(t.src, i) * coef.x * coef.y);
        }
        k -= int32_t(gridDim.x);
        if (k < 0) return;
        t = tiles[k];
    }
}

using ScaleKernel = void (*)(const Tile*, int32_t, Clip);

template <int SRC>
ScaleKernel scale_kernel(int32_t dst) {
    switch (dst) {
        case ADAMW_DTYPE_BF16: return grad_scale_kernel<SRC, ADAMW_DTYPE_BF16>;
        case ADAMW_DTYPE_FP16: return grad_scale_kernel<SRC, ADAMW_DTYPE_FP16>;
        default: return grad_scale_kernel<SRC, ADAMW_DTYPE_FP32>;
    }
}

ScaleKernel scale_kernel(int32_t src, int32_t dst) {
    switch (src) {
        case ADAMW_DTYPE_BF16: return scale_kernel<ADAMW_DTYPE_BF16>(dst);
        case ADAMW_DTYPE_FP16: return scale_kernel<ADAMW_DTYPE_FP16>(dst);
        default: return scale_kernel<ADAMW_DTYPE_FP32>(dst);
    }
}

// Makes a device current for the scope, restoring the caller's.
struct OnDevice {
    int prev = -1;
    bool ok = true;
    explicit OnDevice(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess; else prev = -1;
    }
    ~OnDevice() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

int check_list(const adamw_grad_t* g, int32_t n) {
    if (n < 0 || (n > 0 && !g)) return ADAMW_ERR_INVALID_ARG;
    for (int32_t k = 0; k < n; ++k) {
        const int s = dtype_size(g[k].src_dtype), d = dtype_size(g[k].dst_dtype);
        if (g[k].numel < 0 || s == 0 || (g[k].dst && d == 0)) return ADAMW_ERR_INVALID_ARG;
        if (g[k].numel == 0) continue;
        if (!g[k].src) return ADAMW_ERR_INVALID_ARG;
        if (g[k].numel > (int64_t(1) << 40)) return ADAMW_ERR_TOO_LARGE;
        if (!aligned(g[k].src, uintptr_t(s)) || (g[k].dst && !aligned(g[k].dst, uintptr_t(d))))
            return ADAMW_ERR_MISALIGNED;
        if (!g[k].dst) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(g[k].src), b = reinterpret_cast<uintptr_t>(g[k].dst);
        if (a == b) {
            if (g[k].src_dtype != g[k].dst_dtype) return ADAMW_ERR_INVALID_ARG;
        } else if (a < b + uintptr_t(g[k].numel) * uintptr_t(d) && b < a + uintptr_t(g[k].numel) * uintptr_t(s)) {
            return ADAMW_ERR_INVALID_ARG;
        }
    }
    return ADAMW_OK;
}

// No buffer of an entry reaches into another entry's: the norm would count a
// gradient twice, or two CTAs write the same place.
int check_apart(const adamw_grad_t* g, int32_t n) {
    struct Span {
        uintptr_t begin, end;
    };
    std::vector<Span> spans;
    for (int32_t k = 0; k < n; ++k) {
        if (g[k].numel == 0) continue;
        const void* buffers[] = {g[k].src, g[k].dst == g[k].src ? nullptr : g[k].dst};
        const int32_t types[] = {g[k].src_dtype, g[k].dst_dtype};
        for (int b = 0; b < 2; ++b) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(buffers[b]);
            if (at) spans.push_back({at, at + uintptr_t(g[k].numel) * uintptr_t(dtype_size(types[b]))});
        }
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
    for (size_t k = 1; k < spans.size(); ++k)
        if (spans[k].begin < spans[k - 1].end) return ADAMW_ERR_INVALID_ARG;
    return ADAMW_OK;
}

// The device can dereference p (as adamw_plan_create checks).
int check_access(const void* p, int device, int pageable) {
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        adamw::set_cuda_error("cudaPointerGetAttributes", cudaGetErrorString(cudaGetLastError()));
        return ADAMW_ERR_NOT_ACCESSIBLE;
    }
    bool ok;
    switch (a.type) {
        case cudaMemoryTypeDevice: ok = a.device == device; break;
        case cudaMemoryTypeManaged: ok = true; break;
        case cudaMemoryTypeHost: ok = a.devicePointer == p; break;
        default: ok = pageable != 0; break;
    }
    return ok ? ADAMW_OK : ADAMW_ERR_NOT_ACCESSIBLE;
}

}  // namespace

struct adamw_clip_plan {
    int device = 0;
    int32_t n_tiles = 0;
    int32_t norm_grid[2] = {0, 0};   // by ADAMW_NORM_*
    // the tiles to scale, by their pair of types
    struct Group {
        ScaleKernel kernel;
        int32_t first, n, grid;
    };
    std::vector<Group> groups;
    void* block = nullptr;           // tiles, then partial values
    Tile* tiles = nullptr;
    Partial* partial = nullptr;
};

namespace {

int create(const adamw_grad_t* table, int32_t n, adamw_clip_plan* P) {
    if (!launched(cudaGetDevice(&P->device), "cudaGetDevice")) return ADAMW_ERR_CUDA;
    int pageable = 0, sms = 0;
    if (!launched(cudaDeviceGetAttribute(&pageable, cudaDevAttrPageableMemoryAccess, P->device), "cudaDeviceGetAttribute") ||
        !launched(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, P->device), "cudaDeviceGetAttribute"))
        return ADAMW_ERR_CUDA;
    int64_t total = 0;
    for (int32_t k = 0; k < n; ++k) {
        const adamw_grad_t& g = table[k];
        if (g.numel == 0) continue;
        int rc = check_access(g.src, P->device, pageable);
        if (rc == ADAMW_OK && g.dst) rc = check_access(g.dst, P->device, pageable);
        if (rc != ADAMW_OK) return rc;
        total += g.numel;
        if (total > kMaxTiles * kMaxTile) return ADAMW_ERR_TOO_LARGE;   // before it can overflow
    }
    int64_t tile = kMaxTile;
    while (tile > kMinTile && total < tile * sms * 2) tile /= 2;
    // no device holds a trillion gradients: a size that was meant otherwise
    if (total / tile + n > kMaxTiles) return ADAMW_ERR_TOO_LARGE;
    // pair by pair of types, tensors that are only read first
    std::vector<Tile> tiles;
    for (int pair = -1; pair < 9; ++pair) {
        const size_t first = tiles.size();
        for (int32_t k = 0; k < n; ++k) {
            const adamw_grad_t& g = table[k];
            if (g.numel == 0 || (g.dst ? g.src_dtype * 3 + g.dst_dtype : -1) != pair) continue;
            const int s = dtype_size(g.src_dtype), d = g.dst ? dtype_size(g.dst_dtype) : 0;
            Tile t = {};
            t.src_type = g.src_dtype;
            t.vector = aligned(g.src, 16) && aligned(g.dst, 16);
            for (int64_t at = 0; at < g.numel; at += tile) {
                t.src = static_cast<const char*>(g.src) + at * s;
                t.dst = g.dst ? static_cast<char*>(g.dst) + at * d : nullptr;
                t.len = int32_t(g.numel - at < tile ? g.numel - at : tile);
                tiles.push_back(t);
            }
        }
        const int32_t count = int32_t(tiles.size() - first);
        if (pair < 0 || count == 0) continue;
        ScaleKernel kernel = scale_kernel(pair / 3, pair % 3);
        int occ = 0;
        if (!launched(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, kThreads, 0), "occupancy"))
            return ADAMW_ERR_CUDA;
        const int32_t grid = sms * (occ > 0 ? occ : 1);
        P->groups.push_back({kernel, int32_t(first), count, grid < count ? grid : count});
    }
    P->n_tiles = int32_t(tiles.size());
    int occ[2] = {0, 0};
    if (!launched(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ[0], grad_norm_kernel<false>, kThreads, 0), "occupancy") ||
        !launched(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ[1], grad_norm_kernel<true>, kThreads, 0), "occupancy"))
        return ADAMW_ERR_CUDA;
    for (int k = 0; k < 2; ++k) {
        int64_t g = int64_t(sms) * (occ[k] > 0 ? occ[k] : 1);
        if (g > kMaxGrid) g = kMaxGrid;
        // one CTA at least: an empty list's norm is 0
        P->norm_grid[k] = int32_t(g < P->n_tiles ? g : P->n_tiles > 0 ? P->n_tiles : 1);
    }
    const size_t tile_bytes = sizeof(Tile) * tiles.size();
    if (!launched(cudaMalloc(&P->block, tile_bytes + kMaxGrid * sizeof(Partial)), "cudaMalloc"))
        return ADAMW_ERR_CUDA;
    P->tiles = static_cast<Tile*>(P->block);
    P->partial = reinterpret_cast<Partial*>(static_cast<char*>(P->block) + tile_bytes);
    const bool ok = (tiles.empty() || launched(cudaMemcpy(P->tiles, tiles.data(), tile_bytes, cudaMemcpyHostToDevice), "cudaMemcpy(tiles)")) &&
                    launched(cudaStreamSynchronize(nullptr), "cudaStreamSynchronize");
    return ok ? ADAMW_OK : ADAMW_ERR_CUDA;
}

}  // namespace

extern "C" int adamw_clip_plan_create(const adamw_grad_t* host_table, int32_t n, adamw_clip_plan_t* out) {
    if (!out) return ADAMW_ERR_INVALID_ARG;
    *out = nullptr;
    int rc = check_list(host_table, n);
    if (rc != ADAMW_OK) return rc;
    adamw_clip_plan* P = new (std::nothrow) adamw_clip_plan;
    if (!P) return ADAMW_ERR_TOO_LARGE;
    try {
        rc = check_apart(host_table, n);
        if (rc == ADAMW_OK) rc = create(host_table, n, P);
    } catch (const std::exception&) {  // the host has no room for a table
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

extern "C" int adamw_clip_grads(adamw_clip_plan_t plan, float max_norm, int32_t norm,
                                adamw_clip_result_t* result, adamw_stream_t stream) {
    if (!plan || !result || !(max_norm > 0.0f) || (norm != ADAMW_NORM_L2 && norm != ADAMW_NORM_MAX))
        return ADAMW_ERR_INVALID_ARG;
    if (!aligned(result, 16)) return ADAMW_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    OnDevice guard(plan->device);
    if (!guard.ok) {
        adamw::set_cuda_error("cudaSetDevice", cudaGetErrorString(cudaGetLastError()));
        return ADAMW_ERR_CUDA;
    }
    auto kernel = norm == ADAMW_NORM_MAX ? grad_norm_kernel<true> : grad_norm_kernel<false>;
    const int32_t grid = plan->norm_grid[norm];
    if (!launched(launch(kernel, uint32_t(grid), kThreads, 1, 0, st, static_cast<const Tile*>(plan->tiles),
                         plan->n_tiles, plan->partial), "grad_norm launch"))
        return ADAMW_ERR_CUDA;
    Clip clip = {plan->partial, grid, norm, max_norm, result};
    if (plan->groups.empty())
        return launched(launch(clip_result_kernel, 1u, kThreads, 1, 0, st, clip), "clip_result launch")
                   ? ADAMW_OK : ADAMW_ERR_CUDA;
    for (auto g = plan->groups.rbegin(); g != plan->groups.rend(); ++g) {
        if (!launched(launch(g->kernel, uint32_t(g->grid), kThreads, 1, 0, st,
                             static_cast<const Tile*>(plan->tiles + g->first), g->n, clip), "grad_scale launch"))
            return ADAMW_ERR_CUDA;
        clip.result = nullptr;   // written
    }
    return ADAMW_OK;
}

extern "C" int adamw_clip_plan_destroy(adamw_clip_plan_t plan) {
    if (!plan) return ADAMW_OK;
    OnDevice guard(plan->device);
    bool ok = guard.ok;
    if (plan->block) {
        ok = ok && launched(cudaDeviceSynchronize(), "cudaDeviceSynchronize");
        ok = launched(cudaFree(plan->block), "cudaFree") && ok;
    }
    delete plan;
    return ok ? ADAMW_OK : ADAMW_ERR_CUDA;
}
