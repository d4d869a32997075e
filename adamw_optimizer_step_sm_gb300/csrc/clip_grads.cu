// clip_grads.cu -- the global norm of a list of gradients of several types and
// the clip by it.
//
// Bound by HBM: the list is read for the norm and, its coefficient known only
// after the last element, read again to be scaled (a list that fits the
// 129 MB L2 comes from there the second time).
#include <new>
#include <vector>

#include "losses_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Elements of a tile, the piece of a tensor that a CTA takes at a time: the
// largest that gives every resident CTA one, in [2048, 16384].
constexpr int kMaxTile = 16384, kMinTile = 2048;
constexpr int kNormUnroll = 8;   // 16-byte vectors in flight per thread
constexpr int kScaleVecs = 8;    // likewise, when scaling
constexpr int kMaxGrid = 1216;   // CTAs of the norm pass at most: its partials

struct alignas(16) Tile {
    const char* src;
    char* dst;
    int32_t len;
    int32_t src_type;
    int32_t vector;   // both 16-byte aligned
    int32_t pad_;
};
static_assert(sizeof(Tile) == 32, "tile layout");

// The coefficient in two factors, the second a power of two: a coefficient
// below fp32's normal range (a norm above 1e38 times the limit) keeps its
// digits in the first.  {1, 1} when nothing is scaled.
struct ClipState {
    uint32_t ticket;
    int32_t pad_;
    float2 coef;
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

template <bool MAX>
struct NormOf;
template <>
struct NormOf<false> {
    using Acc = SquareSum;
    __device__ static double value(const Acc& a) { return double(a.sum.hi) + double(a.sum.lo) + a.rare; }
    __device__ static double join(double a, double b) { return a + b; }
    __device__ static double norm(double a) { return sqrt(a); }
};
template <>
struct NormOf<true> {
    using Acc = MaxBits;
    __device__ static double value(const Acc& a) { return double(__uint_as_float(a.bits)); }
    __device__ static double join(double a, double b) { return a != a || a > b ? a : b; }
    __device__ static double norm(double a) { return a; }
};

// The CTA's joined value, in thread 0.
template <bool MAX>
__device__ __forceinline__ double cta_join(double v) {
    using N = NormOf<MAX>;
    __shared__ double part[kWarps];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = N::join(v, __shfl_down_sync(0xffffffffu, v, d));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kWarps; ++w) v = N::join(v, part[w]);
    return v;
}

// The norm: tiles dealt round-robin to a resident grid, each CTA's value left
// in partial[]; the last CTA to finish joins them in order and writes the
// result.
template <bool MAX>
__global__ void __launch_bounds__(kThreads, 4)
grad_norm_kernel(const Tile* tiles, int32_t n, float max_norm, double* partial, ClipState* state,
                 adamw_clip_result_t* result) {
    using N = NormOf<MAX>;
    dependency_trigger();
    dependency_wait();
    typename N::Acc acc = {};
    for (int32_t k = blockIdx.x; k < n; k += gridDim.x) {
        const Tile t = tiles[k];
        switch (t.src_type) {
            case ADAMW_DTYPE_BF16: norm_tile<ADAMW_DTYPE_BF16>(t, acc); break;
            case ADAMW_DTYPE_FP16: norm_tile<ADAMW_DTYPE_FP16>(t, acc); break;
            default: norm_tile<ADAMW_DTYPE_FP32>(t, acc); break;
        }
    }
    __shared__ bool last;
    double v = cta_join<MAX>(N::value(acc));
    if (threadIdx.x == 0) {
        partial[blockIdx.x] = v;
        __threadfence();
        last = atomicAdd(&state->ticket, 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    v = 0.0;
    for (uint32_t b = threadIdx.x; b < gridDim.x; b += kThreads) v = N::join(v, __ldcg(&partial[b]));
    v = cta_join<MAX>(v);
    if (threadIdx.x == 0) {
        const double norm = N::norm(v);
        const bool finite = isfinite(norm);
        const double coef = double(max_norm) / (norm + 1e-6);
        adamw_clip_result_t r;
        r.norm = float(norm);
        r.coef = finite && coef < 1.0 ? float(coef) : 1.0f;
        r.nonfinite = finite ? 0 : 1;
        r.pad_ = 0;
        *result = r;
        const bool tiny = r.coef < 0x1p-100f;   // by at most 2^-160 or so
        state->coef = make_float2(tiny ? float(coef * 0x1p64) : r.coef, tiny ? 0x1p-64f : 1.0f);
        state->ticket = 0;
    }
}

// dst = coef * src for the tiles [first, first + n), all of the kernel's pair
// of types.  In reverse: those that the norm pass read last are the likeliest
// to be in L2 still.
template <int SRC, int DST>
__global__ void __launch_bounds__(kThreads, 4)
grad_scale_kernel(const Tile* tiles, int32_t n, const ClipState* state) {
    using S = Elem<SRC>;
    using D = Elem<DST>;
    // elements per step: whole 16-byte vectors on both sides
    constexpr int K = S::kVec > D::kVec ? S::kVec : D::kVec;
    constexpr int kIn = K / S::kVec, kOut = K / D::kVec;
    constexpr int U = kScaleVecs / kIn;
    dependency_trigger();
    dependency_wait();
    const float2 coef = state->coef;
    auto scaled = [&](uint4 (&v)[kIn], char* dst) {
        float x[K];
#pragma unroll
        for (int j = 0; j < kIn; ++j) S::unpack(v[j], x + j * S::kVec);
#pragma unroll
        for (int j = 0; j < K; ++j) x[j] = x[j] * coef.x * coef.y;
#pragma unroll
        for (int j = 0; j < kOut; ++j) store16(dst + j * 16, D::pack(x + j * D::kVec));
    };
    for (int32_t k = n - 1 - int32_t(blockIdx.x); k >= 0; k -= gridDim.x) {
        const Tile t = tiles[k];
        if (coef.x == 1.0f && t.dst == t.src) continue;
        int done = 0;
        if (t.vector) {
            const int steps = t.len / K;
            int base = threadIdx.x;
            for (; base + (U - 1) * kThreads < steps; base += U * kThreads) {
                uint4 v[U][kIn];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < kIn; ++j)
                        v[u][j] = load16(t.src + ((base + u * kThreads) * kIn + j) * 16);
#pragma unroll
                for (int u = 0; u < U; ++u) scaled(v[u], t.dst + (base + u * kThreads) * kOut * 16);
            }
            for (; base < steps; base += kThreads) {
                uint4 v[kIn];
#pragma unroll
                for (int j = 0; j < kIn; ++j) v[j] = load16(t.src + (base * kIn + j) * 16);
                scaled(v, t.dst + base * kOut * 16);
            }
            done = steps * K;
        }
        for (int i = done + threadIdx.x; i < t.len; i += kThreads)
            D::store(t.dst, i, S::load(t.src, i) * coef.x * coef.y);
    }
}

using ScaleKernel = void (*)(const Tile*, int32_t, const ClipState*);

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
        if (g[k].numel > (int64_t(1) << 48)) return ADAMW_ERR_TOO_LARGE;
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
    void* block = nullptr;           // tiles, then partials, then the state
    Tile* tiles = nullptr;
    double* partial = nullptr;
    ClipState* state = nullptr;
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
    }
    int64_t tile = kMaxTile;
    while (tile > kMinTile && total < tile * sms * 4) tile /= 2;
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
        if (int64_t(tiles.size()) > kMaxCount - kMaxGrid) return ADAMW_ERR_TOO_LARGE;
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
    if (!launched(cudaMalloc(&P->block, tile_bytes + kMaxGrid * sizeof(double) + sizeof(ClipState)), "cudaMalloc"))
        return ADAMW_ERR_CUDA;
    P->tiles = static_cast<Tile*>(P->block);
    P->partial = reinterpret_cast<double*>(static_cast<char*>(P->block) + tile_bytes);
    P->state = reinterpret_cast<ClipState*>(P->partial + kMaxGrid);
    const bool ok = (tiles.empty() || launched(cudaMemcpy(P->tiles, tiles.data(), tile_bytes, cudaMemcpyHostToDevice), "cudaMemcpy(tiles)")) &&
                    launched(cudaMemset(P->state, 0, sizeof(ClipState)), "cudaMemset") &&
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
        rc = create(host_table, n, P);
    } catch (const std::bad_alloc&) {  // the host has no room for the tile table
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
    if (!launched(launch(kernel, uint32_t(plan->norm_grid[norm]), kThreads, 1, 0, st, static_cast<const Tile*>(plan->tiles), plan->n_tiles,
                         max_norm, plan->partial, plan->state, result), "grad_norm launch"))
        return ADAMW_ERR_CUDA;
    for (auto g = plan->groups.rbegin(); g != plan->groups.rend(); ++g)
        if (!launched(launch(g->kernel, uint32_t(g->grid), kThreads, 1, 0, st,
                             static_cast<const Tile*>(plan->tiles + g->first), g->n,
                             static_cast<const ClipState*>(plan->state)), "grad_scale launch"))
            return ADAMW_ERR_CUDA;
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
