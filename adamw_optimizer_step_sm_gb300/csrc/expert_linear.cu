// expert_linear.cu -- products grouped by expert, and the gradient of the
// experts' matrices.
//
// The sizes of the groups are device data: every CTA reads the offsets, and
// works out the list of tiles from them, so that no call waits for the host.
//
// Bounds and figures (bf16, weights of 8192 x 2048).  Many tokens: the tensor
// cores under the power limit; 20480 tokens of 16 experts 363 us a product and as
// much for each gradient (1.9 PFLOP/s). Few tokens an expert: HBM, the weights read
// once; 64 tokens in each of 16 experts 92 us (5.9 TB/s), 256 in each 103 us.
// Between them rows that do not fill a tile: 384 in each of 16 take 155 us of 108 that
// their products need. Loads to L2 ahead of the ring (16 steps) made these 10 to 30 %
// slower and are not kept. Up to 16 tokens: stream_kernel.
#include "adamw_matrix.h"
#include "tensor_product.cuh"

namespace {

constexpr int kMaxExperts = 1024;

// Ends of the groups of rows: [0, first offset) and [last offset, rows) belong
// to no expert and are the first and the last group.
//   bounds[g] .. bounds[g + 1]: rows of group g = 0 .. experts + 1
//   tiles[g]: tiles before group g
struct Groups {
    int32_t bounds[kMaxExperts + 3];
    int32_t tiles[kMaxExperts + 3];
};

// One warp.  row_tile: rows of a tile; per: tiles for each of them.
__device__ void build_groups(Groups* g, const int64_t* offsets, int32_t experts, int64_t rows, int32_t row_tile, int32_t per) {
    const int lane = int(threadIdx.x) % 32;
    int32_t top = 0, sum = 0;   // the largest offset, and the tiles, so far
    if (lane == 0) g->bounds[0] = 0;
    for (int base = 0; base <= experts + 1; base += 32) {
        const int i = base + lane;
        int32_t end = 0;   // of group i
        if (i <= experts) {
            const int64_t v = offsets[i];
            end = int32_t(v < 0 ? 0 : v > rows ? rows : v);
        } else {
            end = int32_t(rows);
        }
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int32_t o = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d && o > end) end = o;
        }
        if (top > end) end = top;
        int32_t begin = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) begin = top;
        int32_t n = i <= experts + 1 ? (end - begin + row_tile - 1) / row_tile * per : 0;
        const int32_t mine = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int32_t o = __shfl_up_sync(0xffffffffu, n, d);
            if (lane >= d) n += o;
        }
        if (i <= experts + 1) {
            g->bounds[i + 1] = end;
            g->tiles[i] = sum + n - mine;
            if (i == experts + 1) g->tiles[i + 1] = sum + n;
        }
        top = __shfl_sync(0xffffffffu, end, 31);
        sum += __shfl_sync(0xffffffffu, n, 31);
    }
}

// The group that tile t is of.
__device__ __forceinline__ int group_of(const Groups* g, int32_t experts, int32_t t) {
    int low = 0, high = experts + 2;   // tiles[low] <= t < tiles[high]
    while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (g->tiles[mid] <= t) low = mid; else high = mid;
    }
    return low;
}

// Rows of any type.
struct RowsAt {
    char* data;
    int64_t ld;
    int32_t cols, dtype;
    int32_t vector;   // kAnyRows, ...
};

// The rows from (row, col) on.
__device__ __forceinline__ RowsAt part_of(RowsAt r, int64_t row, int32_t col) {
    r.data += (row * r.ld + col) * (r.dtype == ADAMW_DTYPE_FP32 ? 4 : 2);
    r.cols -= col;
    return r;
}

// Tile (m, n) number i of a group of tm x tn: bands of eight tiles of rows, so
// that tiles worked on at a time share rows of both operands in L2.
__device__ __forceinline__ void banded(int32_t i, int32_t tm, int32_t tn, int32_t* m, int32_t* n) {
    const int32_t band = i / (8 * tn), left = tm - band * 8, h = left < 8 ? left : 8;
    i -= band * 8 * tn;
    *m = band * 8 + i % h;
    *n = i / h;
}

// Results of 16 bits at rows of whole 16 bytes leave by TMA, in blocks of 32 rows
// of 64 columns through a buffer of the warp's (sectors by threads made four
// times the requests: the gradient of 120 matrices of 768 x 2048 from 16320 tokens
// 134 us, staged 79). `rows`: of the block; a block with fewer than 32 goes
// by sectors.
template <int BUFFERS>
__device__ __forceinline__ void store_block(const CUtensorMap* map, bool bf16, const RowsAt& out, int x, int y, int z, int rows, int c,
                                            Staged& s, bool any) {
    if (rows >= 32) {
        unsigned char* buffer = BUFFERS > 1 && s.turn ? s.two : s.one;
        s.turn ^= 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v[32];
            load_acc(s.acc + uint32_t(c + half * 32), any, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *unit_of(buffer, s.lane, half * 4 + j) =
                    bf16 ? Elem<ADAMW_DTYPE_BF16>::pack(v + j * 8) : Elem<ADAMW_DTYPE_FP16>::pack(v + j * 8);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (elected()) {
            store_box(map, x, y, z, smem_addr(buffer));
            if (BUFFERS > 1) stores_read_but_one(); else stores_read();   // the next buffer is free
        }
        __syncwarp();
        return;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int n = out.cols - c - half * 32;
        if (n <= 0) break;
        float v[32];
        load_acc(s.acc + uint32_t(c + half * 32), any, v);
        if (s.lane < rows)
            store_row(out.data + (int64_t(s.row + s.lane) * out.ld + c + half * 32) * 2, out.dtype, v, n, out.vector == kSectorRows);
    }
}

// y = x w^T by groups of rows: A is x (K-major), B the expert's matrix.
template <class S, bool STAGED>
struct ExpertRows {
    struct Params {
        CUtensorMap x, w, result;
        const int64_t* offsets;
        int64_t rows;
        int32_t experts, k, tiles_n;
        bool is_bf16, w_mn, shared;   // shared: one matrix for all experts
        RowsAt y;
    };
    static constexpr bool kTail = false, kParts = false;
    static constexpr size_t kTable = sizeof(Groups);
    static constexpr uint32_t kRing = 196608;
    static constexpr int kWarps = 4;
    static constexpr uint32_t kStaging = 4096;
    static constexpr bool kStaged = STAGED;
    struct Out {
        RowsAt y;       // from the first row and column of the CTA's part
        int32_t rows;   // of the group, from there (0 or less: none)
        int32_t row, col;
    };
    __device__ static bool bf16(const Params& p) { return p.is_bf16; }
    __device__ static void prepare(const Params& p, unsigned char* table) {
        if (threadIdx.x < 32)
            build_groups(reinterpret_cast<Groups*>(table), p.offsets, p.experts, p.rows, S::kRows, p.tiles_n);
    }
    __device__ static int tiles(const Params& p, const unsigned char* table) {
        return reinterpret_cast<const Groups*>(table)->tiles[p.experts + 2];
    }
    __device__ static int find(const Params& p, const unsigned char* table, int t, int32_t* m, int32_t* n) {
        const Groups* g = reinterpret_cast<const Groups*>(table);
        const int k = group_of(g, p.experts, t);
        banded(t - g->tiles[k], (g->bounds[k + 1] - g->bounds[k] + S::kRows - 1) / S::kRows, p.tiles_n, m, n);
        return k;
    }
    __device__ static void loads(const Params& p, const unsigned char* table, int t, TileLoads& w) {
        int32_t m, n;
        const int k = find(p, table, t, &m, &n);
        const Groups* g = reinterpret_cast<const Groups*>(table);
        w.a = &p.x;
        w.b = &p.w;
        w.a_at = g->bounds[k] + m * S::kRows;
        w.b_at = n * S::kCols;
        w.a_z = 0;
        w.b_z = p.shared ? 0 : k - 1;
        w.k_at = 0;
        w.k_len = k == 0 || k == p.experts + 1 ? 0 : p.k;
        w.a_mn = false;
        w.b_mn = p.w_mn;
    }
    template <class>
    __device__ static Out out(const Params& p, const unsigned char* table, int t, uint32_t rank) {
        int32_t m, n;
        const int k = find(p, table, t, &m, &n);
        const Groups* g = reinterpret_cast<const Groups*>(table);
        const int64_t row = int64_t(g->bounds[k]) + int64_t(m) * S::kRows + int64_t(rank) * kRowsOfCta;
        return {part_of(p.y, row, n * S::kCols), int32_t(g->bounds[k + 1] - row), int32_t(row), n * S::kCols};
    }
    __device__ static bool wanted(const Params&, const Out& o, int row, int col) { return row < o.rows && col < o.y.cols; }
    __device__ static void begin(const Params&, const Out&, Staged&, int) {}
    __device__ static void gave_up(const Params&) {}
    __device__ static bool pretend(const Params&) { return false; }
    __device__ static bool finish(const Params& p, const Out& o, Staged& s, bool any) {
        for (int c = s.col; c < s.end && wanted(p, o, s.row, c); c += kBlock64)
            store_block<1>(&p.result, o.y.dtype == ADAMW_DTYPE_BF16, o.y, o.col + c, o.row + s.row, 0, o.rows - s.row, c, s, any);
        return true;
    }
    __device__ static bool scalar(const Out& o) { return !o.y.vector; }
    __device__ static void store(const Params& p, const Out& o, int row, int col, float (&v)[32]) {
        if (o.y.vector && row < o.rows)
            store_row(o.y.data + (row * o.y.ld + col) * (o.y.dtype == ADAMW_DTYPE_FP32 ? 4 : 2), o.y.dtype, v, o.y.cols - col,
                      o.y.vector == kSectorRows);
    }
    __device__ static void store_one(const Params& p, const Out& o, int row, int col, float v) {
        if (wanted(p, o, row, col)) store_as(o.y.data, row * o.y.ld + col, o.y.dtype, v);
    }
};

// dw[e] = dy^T x over the expert's rows: both operands MN-major.
// STAGED: buffers of a warp for results that leave by TMA, 0 for those that do not.
template <class S, bool ADD, int STAGED>
struct ExpertOuter {
    static_assert(!ADD || STAGED == 0, "what is added to is read");
    struct Params {
        CUtensorMap dy, x, result;
        const int64_t* offsets;
        int64_t rows;
        int32_t experts, n, tiles_m, tiles_n;
        bool is_bf16;
        int64_t stride;   // of dw's matrices
        RowsAt dw;
    };
    static constexpr bool kTail = true, kParts = false;
    static constexpr size_t kTable = sizeof(Groups);
    static constexpr uint32_t kRing = STAGED < 2 ? 196608 : S::kStageBytes > 32768 ? 147456 : 163840;
    static constexpr int kWarps = 4;
    static constexpr uint32_t kStaging = STAGED < 2 ? 4096 : 8192;
    static constexpr bool kStaged = STAGED > 0;
    struct Out {
        RowsAt dw;      // from the first row and column of the CTA's part
        int32_t rows;   // of dw, from there
        int32_t row, col, expert;
    };
    __device__ static bool bf16(const Params& p) { return p.is_bf16; }
    __device__ static void prepare(const Params& p, unsigned char* table) {
        if (threadIdx.x < 32) build_groups(reinterpret_cast<Groups*>(table), p.offsets, p.experts, p.rows, 1, 0);
    }
    __device__ static int tiles(const Params& p, const unsigned char*) { return p.experts * p.tiles_m * p.tiles_n; }
    __device__ static void loads(const Params& p, const unsigned char* table, int t, TileLoads& w) {
        const int32_t per = p.tiles_m * p.tiles_n, e = t / per;
        int32_t m, n;
        banded(t - e * per, p.tiles_m, p.tiles_n, &m, &n);
        const Groups* g = reinterpret_cast<const Groups*>(table);
        w.a = &p.dy;
        w.b = &p.x;
        w.a_at = m * S::kRows;
        w.b_at = n * S::kCols;
        w.a_z = w.b_z = 0;
        w.k_at = g->bounds[e + 1];
        w.k_len = g->bounds[e + 2] - g->bounds[e + 1];
        w.a_mn = w.b_mn = true;
    }
    template <class>
    __device__ static Out out(const Params& p, const unsigned char* table, int t, uint32_t rank) {
        const int32_t per = p.tiles_m * p.tiles_n, e = t / per;
        int32_t m, n;
        banded(t - e * per, p.tiles_m, p.tiles_n, &m, &n);
        const Groups* g = reinterpret_cast<const Groups*>(table);
        RowsAt r = p.dw;
        r.data += e * p.stride * (r.dtype == ADAMW_DTYPE_FP32 ? 4 : 2);
        const int32_t row = m * S::kRows + int32_t(rank) * kRowsOfCta;
        // nothing to add: the sums stay as they are
        const bool skip = ADD && g->bounds[e + 2] == g->bounds[e + 1];
        return {part_of(r, row, n * S::kCols), skip ? 0 : p.n - row, row, n * S::kCols, e};
    }
    __device__ static bool wanted(const Params&, const Out& o, int row, int col) { return row < o.rows && col < o.dw.cols; }
    __device__ static void begin(const Params&, const Out&, Staged&, int) {}
    __device__ static void gave_up(const Params&) {}
    __device__ static bool pretend(const Params&) { return false; }
    __device__ static bool finish(const Params& p, const Out& o, Staged& s, bool any) {
        // rows beyond dw's end are left out by TMA
        for (int c = s.col; c < s.end && wanted(p, o, s.row, c); c += kBlock64)
            store_block<STAGED>(&p.result, o.dw.dtype == ADAMW_DTYPE_BF16, o.dw, o.col + c, o.row + s.row, o.expert, 32, c, s, any);
        return true;
    }
    __device__ static bool scalar(const Out& o) { return !o.dw.vector; }
    __device__ static void store(const Params& p, const Out& o, int row, int col, float (&v)[32]) {
        if (!o.dw.vector || row >= o.rows) return;
        char* at = o.dw.data + (row * o.dw.ld + col) * (o.dw.dtype == ADAMW_DTYPE_FP32 ? 4 : 2);
        if constexpr (ADD) {
            float sum[32];
            load_row(at, o.dw.dtype, sum, o.dw.cols - col, o.dw.vector == kSectorRows);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += sum[i];
        }
        store_row(at, o.dw.dtype, v, o.dw.cols - col, o.dw.vector == kSectorRows);
    }
    __device__ static void store_one(const Params& p, const Out& o, int row, int col, float v) {
        if (!wanted(p, o, row, col)) return;
        const int64_t at = row * o.dw.ld + col;
        if constexpr (ADD) v += load_as(o.dw.data, at, o.dw.dtype);
        store_as(o.dw.data, at, o.dw.dtype, v);
    }
};

// ------------------------------------------------------------- few tokens --

// The product for a few tokens (decoding): bound by reading the weights of the
// experts that have one, once, at HBM's rate.  A warp has four rows of a matrix,
// a lane every 32nd 16 bytes of them, 128 bytes in flight; up to four tokens
// are multiplied at a time, in fp32, and the lanes' sums joined at the end.  The
// tile kernel streams half as much of zero-padded tokens beside the weights
// and was slower up to kStreamTokens: 8 tokens through 7 of 16 matrices of
// 8192 x 2048 (235 MB) 61 us there, 41 here.
constexpr int kStreamThreads = 256, kStreamRows = 4, kStreamTokens = ADAMW_EXPERT_STREAM_ROWS;

struct StreamParams {
    const uint16_t *x, *w;
    int64_t ldx, ldw, w_stride;
    const int64_t* offsets;
    int64_t rows;
    int32_t experts, n, k;
    RowsAt y;
};

template <int DT, bool VEC, int TOKENS>
__device__ __forceinline__ void stream_rows(const StreamParams& p, const uint16_t* w, int row, int token, int tokens) {
    using E = Elem<DT>;
    const int lane = int(threadIdx.x) % 32;
    const uint16_t* x[TOKENS];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) x[t] = p.x + int64_t(token + (t < tokens ? t : tokens - 1)) * p.ldx;
    const uint16_t* m[kStreamRows];
#pragma unroll
    for (int r = 0; r < kStreamRows; ++r) m[r] = w + int64_t(row + r < p.n ? row + r : p.n - 1) * p.ldw;
    float sum[kStreamRows][TOKENS];
    if (VEC) {
        Pair acc[kStreamRows][TOKENS];
#pragma unroll
        for (int r = 0; r < kStreamRows; ++r)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) acc[r][t] = 0;
        const int vecs = p.k / 8;
        auto take = [&](const uint4 (&q)[kStreamRows], int v) {
            Pair a[kStreamRows][4];
#pragma unroll
            for (int r = 0; r < kStreamRows; ++r) E::pairs(q[r], a[r]);
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) {
                Pair b[4];
                E::pairs(load16(reinterpret_cast<const char*>(x[t] + v * 8)), b);
#pragma unroll
                for (int r = 0; r < kStreamRows; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][t] = fma2(a[r][i], b[i], acc[r][t]);
            }
        };
        int v = lane;
        for (; v + 32 < vecs; v += 64) {
            uint4 q[2][kStreamRows];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < kStreamRows; ++r) q[h][r] = load16(reinterpret_cast<const char*>(m[r] + (v + h * 32) * 8));
            take(q[0], v);
            take(q[1], v + 32);
        }
        if (v < vecs) {
            uint4 q[kStreamRows];
#pragma unroll
            for (int r = 0; r < kStreamRows; ++r) q[r] = load16(reinterpret_cast<const char*>(m[r] + v * 8));
            take(q, v);
        }
#pragma unroll
        for (int r = 0; r < kStreamRows; ++r)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) sum[r][t] = low(acc[r][t]) + high(acc[r][t]);
    } else {
#pragma unroll
        for (int r = 0; r < kStreamRows; ++r)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) sum[r][t] = 0.0f;
#pragma unroll 4
        for (int i = lane; i < p.k; i += 32) {
            float a[kStreamRows];
#pragma unroll
            for (int r = 0; r < kStreamRows; ++r) a[r] = E::load(m[r], i);
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) {
                const float b = E::load(x[t], i);
#pragma unroll
                for (int r = 0; r < kStreamRows; ++r) sum[r][t] = fmaf(a[r], b, sum[r][t]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kStreamRows; ++r)
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            float s = sum[r][t];
#pragma unroll
            for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == (r * TOKENS + t) % 32 && t < tokens && row + r < p.n)
                store_as(p.y.data, int64_t(token + t) * p.y.ld + row + r, p.y.dtype, s);
        }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kStreamThreads, 2) stream_kernel(const __grid_constant__ StreamParams p) {
    __shared__ Groups groups;
    constexpr int kWarps = kStreamThreads / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per = (p.n + kStreamRows - 1) / kStreamRows;   // units of a group with tokens
    if (threadIdx.x < 32) build_groups(&groups, p.offsets, p.experts, p.rows, kStreamTokens, per);
    __syncthreads();
    const int units = groups.tiles[p.experts + 2], lane = int(threadIdx.x) % 32;
    for (int u = int(blockIdx.x) * kWarps + int(threadIdx.x) / 32; u < units; u += int(gridDim.x) * kWarps) {
        const int g = group_of(&groups, p.experts, u), row = (u - groups.tiles[g]) * kStreamRows;
        const int begin = groups.bounds[g], end = groups.bounds[g + 1];
        if (g == 0 || g == p.experts + 1) {   // tokens of no expert
            for (int i = lane; i < (end - begin) * kStreamRows; i += 32)
                if (row + i % kStreamRows < p.n)
                    store_as(p.y.data, int64_t(begin + i / kStreamRows) * p.y.ld + row + i % kStreamRows, p.y.dtype, 0.0f);
            continue;
        }
        const uint16_t* w = p.w + (g - 1) * p.w_stride;
        for (int t = begin; t < end; t += 4) {
            const int n = end - t;
            if (n == 1) stream_rows<DT, VEC, 1>(p, w, row, t, 1);
            else if (n == 2) stream_rows<DT, VEC, 2>(p, w, row, t, 2);
            else stream_rows<DT, VEC, 4>(p, w, row, t, n < 4 ? n : 4);
        }
    }
}

// Batches of matrices of 16-bit elements, at any strides, into rows of `ld`: what
// TMA reads in their place. Up to three in a launch (each costs the host 4 us).
struct PadJob {
    const uint16_t* src;
    uint16_t* dst;
    int64_t total;   // vectors of eight elements
    int64_t row_stride, batch_stride;
    int32_t rows, cols, ld;
};
struct PadJobs {
    PadJob job[3];
    int32_t n;
};

__global__ void __launch_bounds__(256) pad_kernel(const __grid_constant__ PadJobs jobs) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int k = 0; k < jobs.n; ++k) {
        const PadJob& j = jobs.job[k];
        const int32_t per = j.ld / 8;
        for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < j.total; i += int64_t(gridDim.x) * 256) {
            const int64_t line = i / per;
            const int32_t col = int32_t(i - line * per) * 8, row = int32_t(line % j.rows);
            const uint16_t* s = j.src + line / j.rows * j.batch_stride + row * j.row_stride + col;
            uint16_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = col + e < j.cols ? s[e] : 0;
            uint4 w;
            memcpy(&w, v, 16);
            reinterpret_cast<uint4*>(j.dst)[i] = w;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------- host --

bool sixteen(int32_t dt) { return dt == ADAMW_DTYPE_BF16 || dt == ADAMW_DTYPE_FP16; }
constexpr int64_t kMaxSide = int64_t(1) << 30;

int check(const adamw_matrices_t* m, bool operand) {
    if (!m) return ADAMW_ERR_INVALID_ARG;
    if (m->batch < 0 || m->rows < 0 || m->cols < 0 || m->batch_stride < 0 || m->row_stride < 0 || dtype_size(m->dtype) == 0 ||
        (operand && !sixteen(m->dtype)))
        return ADAMW_ERR_INVALID_ARG;
    if (m->rows > kMaxSide || m->cols > kMaxSide || m->row_stride > (int64_t(1) << 40) || m->batch_stride > (int64_t(1) << 40))
        return ADAMW_ERR_TOO_LARGE;
    const bool any = m->batch > 0 && m->rows > 0 && m->cols > 0;
    if (any && !m->data) return ADAMW_ERR_INVALID_ARG;
    if (any && !operand && !apart(*m)) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(m->data, uintptr_t(dtype_size(m->dtype)))) return ADAMW_ERR_MISALIGNED;
    return ADAMW_OK;
}

// One matrix for all of a batch (a stride of 0) is read as the one that it is.
adamw_matrices_t single(adamw_matrices_t m) {
    if (m.batch > 1 && m.batch_stride == 0) m.batch = 1;
    return m;
}
// TMA reads it as it is (its strides are above 0 and below 2^40 bytes).
bool direct(const adamw_matrices_t& m) {
    constexpr int64_t kMost = int64_t(1) << 38;
    return aligned(m.data, 16) && (m.rows <= 1 || (m.row_stride % 8 == 0 && m.row_stride >= m.cols && m.row_stride <= kMost)) &&
           (m.batch <= 1 || (m.batch_stride % 8 == 0 && m.batch_stride > 0 && m.batch_stride <= kMost));
}
int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }
int64_t copy_bytes(const adamw_matrices_t& given) {
    const adamw_matrices_t m = single(given);
    if (direct(m) || m.cols == 0) return 0;
    return (m.batch * m.rows * padded(m.cols) * 2 + 255) / 256 * 256;
}

// The operands where TMA can read them: themselves, or copies in the workspace.
bool readable(adamw_matrices_t* const (&operands)[3], void* workspace, cudaStream_t st) {
    PadJobs jobs;
    memset(&jobs, 0, sizeof jobs);
    char* at = static_cast<char*>(workspace);
    int64_t most = 0;
    for (adamw_matrices_t* m : operands) {
        if (!m || m->batch * m->rows * m->cols == 0) continue;
        *m = single(*m);
        if (direct(*m)) {
            if (m->rows <= 1) m->row_stride = padded(m->cols);
            if (m->batch <= 1) m->batch_stride = m->row_stride * m->rows;
            continue;
        }
        PadJob& j = jobs.job[jobs.n++];
        j.src = static_cast<const uint16_t*>(m->data);
        j.dst = reinterpret_cast<uint16_t*>(at);
        j.ld = int32_t(padded(m->cols));
        j.total = m->batch * m->rows * (j.ld / 8);
        j.row_stride = m->row_stride;
        j.batch_stride = m->batch_stride;
        j.rows = int32_t(m->rows);
        j.cols = int32_t(m->cols);
        most = std::max(most, j.total);
        at += copy_bytes(*m);
        m->data = j.dst;
        m->row_stride = j.ld;
        m->batch_stride = j.ld * m->rows;
    }
    if (jobs.n == 0) return true;
    const int64_t want = (most + 255) / 256;
    return launched(launch(pad_kernel, uint32_t(want < 152 * 8 ? want : 152 * 8), 256, 1, 0, st, jobs), "pad launch");
}

// rows: what a CTA loads of a K-major operand at a time.
bool map_of(CUtensorMap* map, const adamw_matrices_t& m, bool mn, int rows) {
    return tensor_map(map, m.dtype == ADAMW_DTYPE_BF16, m.data, m.batch, m.rows, m.cols, m.row_stride, m.batch_stride,
                      mn ? kStepK : rows);
}

RowsAt rows_of(const adamw_matrices_t& m) {
    return {static_cast<char*>(m.data), m.row_stride, int32_t(m.cols), m.dtype, rows_at(m)};
}

template <class P>
cudaError_t units_of(TileUnits* u) {
    static thread_local int known = -1;
    static thread_local TileUnits units;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (known != device) {
        if ((e = cudaFuncSetAttribute(tile_kernel<P, PairTile>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      int(tile_smem<P>()))) != cudaSuccess) return e;
        if ((e = tile_units<P>(&units)) != cudaSuccess) return e;
        known = device;
    }
    *u = units;
    return cudaSuccess;
}

template <class P, class S>
bool run(const typename P::Params& p, int64_t tiles, int units, cudaStream_t st) {
    const uint32_t grid = uint32_t(tiles < units ? tiles : units) * S::kPair;
    static thread_local int known = -1;
    int device = 0;
    if (!launched(cudaGetDevice(&device), "cudaGetDevice")) return false;
    if (known != device) {
        if (!launched(cudaFuncSetAttribute(tile_kernel<P, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           int(tile_smem<P>())), "cudaFuncSetAttribute"))
            return false;
        known = device;
    }
    return launched(launch(tile_kernel<P, S>, grid, tile_threads<P>(), S::kPair, tile_smem<P>(), st, p), "product launch");
}

int64_t up(int64_t n, int64_t by) { return (n + by - 1) / by; }

// Results that leave by TMA: 16 bits, rows of whole 16 bytes (it writes whole ones: of a row
// that ends inside of one, what lies behind it too), strides that a map takes.
bool stages(const adamw_matrices_t& m) { return sixteen(m.dtype) && m.cols % 8 == 0 && direct(m); }
bool result_map(CUtensorMap* map, adamw_matrices_t m) {
    if (m.rows <= 1) m.row_stride = padded(m.cols);
    if (m.batch <= 1) m.batch_stride = m.row_stride * m.rows;
    return tensor_map(map, m.dtype == ADAMW_DTYPE_BF16, m.data, m.batch, m.rows, m.cols, m.row_stride, m.batch_stride, 32);
}

template <class S, bool STAGED>
int rows_call(const adamw_matrices_t& x, const adamw_matrices_t& w, int64_t experts, bool transposed, const int64_t* offsets,
              const adamw_matrices_t& y, int64_t tiles, int units, cudaStream_t st) {
    using P = ExpertRows<S, STAGED>;
    typename P::Params p;
    memset(&p, 0, sizeof p);
    // sums of nothing read no operand
    if (x.cols > 0 && (!map_of(&p.x, x, false, kRowsOfCta) || !map_of(&p.w, w, transposed, S::kBRows))) return ADAMW_ERR_CUDA;
    if (STAGED && !result_map(&p.result, y)) return ADAMW_ERR_CUDA;
    p.offsets = offsets;
    p.rows = x.rows;
    p.experts = int32_t(experts);
    p.shared = w.batch < experts;
    p.k = int32_t(x.cols);
    p.tiles_n = int32_t(up(y.cols, S::kCols));
    p.is_bf16 = x.dtype == ADAMW_DTYPE_BF16;
    p.w_mn = transposed;
    p.y = rows_of(y);
    return run<P, S>(p, tiles, units, st) ? ADAMW_OK : ADAMW_ERR_CUDA;
}

int stream_call(const adamw_matrices_t& x, const adamw_matrices_t& w, const int64_t* offsets, const adamw_matrices_t& y,
                cudaStream_t st) {
    TileUnits units;
    if (!launched(units_of<ExpertRows<PairTile, true>>(&units), "tile units")) return ADAMW_ERR_CUDA;
    StreamParams p;
    memset(&p, 0, sizeof p);
    p.x = static_cast<const uint16_t*>(x.data);
    p.w = static_cast<const uint16_t*>(w.data);
    p.ldx = x.row_stride;
    p.ldw = w.row_stride;
    p.w_stride = w.batch_stride;
    p.offsets = offsets;
    p.rows = x.rows;
    p.experts = int32_t(w.batch);
    p.n = int32_t(y.cols);
    p.k = int32_t(x.cols);
    p.y = rows_of(y);
    const bool vec = direct(x) && direct(single(w)) && x.cols % 8 == 0, bf16 = x.dtype == ADAMW_DTYPE_BF16;
    const auto kernel = bf16 ? (vec ? stream_kernel<ADAMW_DTYPE_BF16, true> : stream_kernel<ADAMW_DTYPE_BF16, false>)
                             : (vec ? stream_kernel<ADAMW_DTYPE_FP16, true> : stream_kernel<ADAMW_DTYPE_FP16, false>);
    int occ = 0;
    if (!launched(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, kStreamThreads, 0), "occupancy")) return ADAMW_ERR_CUDA;
    // every token in an expert of its own, or in none
    const int64_t most = std::min<int64_t>(x.rows, w.batch + 2) * up(y.cols, kStreamRows);
    const int64_t grid = std::min<int64_t>(up(most, kStreamThreads / 32), int64_t(units.sms) * (occ > 0 ? occ : 1));
    return launched(launch(kernel, uint32_t(grid), kStreamThreads, 1, 0, st, p), "stream launch") ? ADAMW_OK : ADAMW_ERR_CUDA;
}

template <class S, bool ADD, int STAGED>
int outer_call(const adamw_matrices_t& dy, const adamw_matrices_t& x, const int64_t* offsets, const adamw_matrices_t& dw,
               int64_t tiles, int units, cudaStream_t st) {
    using P = ExpertOuter<S, ADD, STAGED>;
    typename P::Params p;
    memset(&p, 0, sizeof p);
    if (x.rows > 0 && (!map_of(&p.dy, dy, true, 0) || !map_of(&p.x, x, true, 0))) return ADAMW_ERR_CUDA;
    if (STAGED && !result_map(&p.result, dw)) return ADAMW_ERR_CUDA;
    p.offsets = offsets;
    p.rows = x.rows;
    p.experts = int32_t(dw.batch);
    p.n = int32_t(dw.rows);
    p.tiles_m = int32_t(up(dw.rows, S::kRows));
    p.tiles_n = int32_t(up(dw.cols, S::kCols));
    p.is_bf16 = x.dtype == ADAMW_DTYPE_BF16;
    p.stride = dw.batch_stride;
    p.dw = rows_of(dw);
    return run<P, S>(p, tiles, units, st) ? ADAMW_OK : ADAMW_ERR_CUDA;
}

}  // namespace

namespace adamw {
int expert_status(int32_t* out) {
    int32_t v = 0;
    const int32_t zero = 0;
    if (!launched(cudaMemcpyFromSymbol(&v, g_tile_status, 4), "cudaMemcpyFromSymbol") ||
        !launched(cudaMemcpyToSymbol(g_tile_status, &zero, 4), "cudaMemcpyToSymbol"))
        return ADAMW_ERR_CUDA;
    *out |= v;
    return ADAMW_OK;
}
}  // namespace adamw

namespace {

int check_rows(const adamw_matrices_t* x, const adamw_matrices_t* w, int32_t transposed, const int64_t* offsets,
               const adamw_matrices_t* y) {
    int rc;
    if ((rc = check(x, true)) != ADAMW_OK || (rc = check(w, true)) != ADAMW_OK || (rc = check(y, false)) != ADAMW_OK) return rc;
    const int64_t n = transposed ? w->cols : w->rows, k = transposed ? w->rows : w->cols;
    if (x->batch != 1 || y->batch != 1 || x->dtype != w->dtype || x->cols != k || y->cols != n || y->rows != x->rows ||
        w->batch < 1 || (transposed != 0 && transposed != 1) || overlap(*y, *x) || overlap(*y, *w))
        return ADAMW_ERR_INVALID_ARG;
    if (w->batch > kMaxExperts) return ADAMW_ERR_TOO_LARGE;
    if (y->rows == 0 || y->cols == 0) return ADAMW_OK;
    if (!offsets) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(offsets, 8)) return ADAMW_ERR_MISALIGNED;
    if ((x->rows / SmallTile::kRows + w->batch + 2) * up(n, SmallTile::kCols) > kMaxCount) return ADAMW_ERR_TOO_LARGE;
    return ADAMW_OK;
}

int check_outer(const adamw_matrices_t* dy, const adamw_matrices_t* x, const int64_t* offsets, const adamw_matrices_t* dw,
                int32_t accumulate) {
    int rc;
    if ((rc = check(dy, true)) != ADAMW_OK || (rc = check(x, true)) != ADAMW_OK || (rc = check(dw, false)) != ADAMW_OK) return rc;
    if (dy->batch != 1 || x->batch != 1 || dy->dtype != x->dtype || dy->rows != x->rows || dw->rows != dy->cols ||
        dw->cols != x->cols || dw->batch < 1 || (accumulate != 0 && accumulate != 1) ||
        overlap(*dw, *dy) || overlap(*dw, *x))
        return ADAMW_ERR_INVALID_ARG;
    if (dw->batch > kMaxExperts) return ADAMW_ERR_TOO_LARGE;
    if (dw->rows == 0 || dw->cols == 0) return ADAMW_OK;
    if (!offsets) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(offsets, 8)) return ADAMW_ERR_MISALIGNED;
    if (dw->batch * up(dw->rows, SmallTile::kRows) * up(dw->cols, SmallTile::kCols) > kMaxCount) return ADAMW_ERR_TOO_LARGE;
    return ADAMW_OK;
}

int check_workspace(int64_t bytes, const void* workspace) {
    if (bytes > 0 && !workspace) return ADAMW_ERR_INVALID_ARG;
    return bytes > 0 && !aligned(workspace, 256) ? ADAMW_ERR_MISALIGNED : ADAMW_OK;
}

// Checked and readable, with something to do.
int launch_rows(const adamw_matrices_t& x, const adamw_matrices_t& w, int64_t experts, bool transposed, const int64_t* offsets,
                const adamw_matrices_t& y, cudaStream_t st) {
    TileUnits units;
    if (!launched(units_of<ExpertRows<PairTile, true>>(&units), "tile units")) return ADAMW_ERR_CUDA;
    const int64_t n = y.cols;
    // the grid covers the most tiles that the groups can have: one partial in each
    const int64_t groups = experts + 2;
    auto most = [&](int rows, int cols) { return (x.rows / rows + groups) * up(n, cols); };
    // what groups of one size would have
    const int64_t each = up(x.rows, experts), used = std::min(experts, x.rows);
    auto likely = [&](int rows, int cols) { return used * up(each, rows) * up(n, cols); };
    const TileChoice choice = {{likely(PairTile::kRows, PairTile::kCols), likely(WideTile::kRows, WideTile::kCols),
                                likely(SmallTile::kRows, SmallTile::kCols)}};
    auto call = [&](auto shape, int u) {
        using S = decltype(shape);
        const int64_t tiles = most(S::kRows, S::kCols);
        return stages(y) ? rows_call<S, true>(x, w, experts, transposed, offsets, y, tiles, u, st)
                         : rows_call<S, false>(x, w, experts, transposed, offsets, y, tiles, u, st);
    };
    switch (choose_shape(choice, up(x.cols, kStepK), units.pairs, units.sms)) {
        case kPairShape: return call(PairTile(), units.pairs);
        case kWideShape: return call(WideTile(), units.sms);
        default: return call(SmallTile(), units.sms);
    }
}

int launch_outer(const adamw_matrices_t& dy, const adamw_matrices_t& x, const int64_t* offsets, const adamw_matrices_t& dw,
                 bool accumulate, cudaStream_t st) {
    TileUnits units;
    if (!launched(units_of<ExpertOuter<PairTile, false, 1>>(&units), "tile units")) return ADAMW_ERR_CUDA;
    auto tiles = [&](int rows, int cols) { return dw.batch * up(dw.rows, rows) * up(dw.cols, cols); };
    const TileChoice choice = {{tiles(PairTile::kRows, PairTile::kCols), tiles(WideTile::kRows, WideTile::kCols),
                                tiles(SmallTile::kRows, SmallTile::kCols)}};
    const int shape = choose_shape(choice, up(up(dy.rows, dw.batch), kStepK), units.pairs, units.sms);
    // Sums over few tokens are bound by the results: two buffers a warp, for a stage
    // of the ring (32 tokens in each of 16 experts, 8192 x 2048: 83 against 106 us;
    // 200 115 / 124; 640 217 / 198).
    const bool brief = dy.rows < dw.batch * 256;
    auto call = [&](auto tile, int u) {
        using S = decltype(tile);
        const int64_t n = choice.tiles[shape];
        return accumulate    ? outer_call<S, true, 0>(dy, x, offsets, dw, n, u, st)
               : !stages(dw) ? outer_call<S, false, 0>(dy, x, offsets, dw, n, u, st)
               : brief       ? outer_call<S, false, 2>(dy, x, offsets, dw, n, u, st)
                             : outer_call<S, false, 1>(dy, x, offsets, dw, n, u, st);
    };
    return shape == kPairShape ? call(PairTile(), units.pairs)
           : shape == kWideShape ? call(WideTile(), units.sms) : call(SmallTile(), units.sms);
}

}  // namespace

extern "C" int64_t adamw_expert_workspace(const adamw_matrices_t* a, const adamw_matrices_t* b) {
    if (check(a, true) != ADAMW_OK || check(b, true) != ADAMW_OK) return 0;
    return copy_bytes(*a) + copy_bytes(*b);
}

extern "C" int adamw_expert_rows(const adamw_matrices_t* x, const adamw_matrices_t* w, int32_t transposed,
                                 const int64_t* offsets, const adamw_matrices_t* y, void* workspace, adamw_stream_t stream) {
    int rc = check_rows(x, w, transposed, offsets, y);
    if (rc != ADAMW_OK || y->rows == 0 || y->cols == 0) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!transposed && x->rows <= kStreamTokens && y->cols < (int64_t(1) << 24)) return stream_call(*x, *w, offsets, *y, st);
    if ((rc = check_workspace(copy_bytes(*x) + copy_bytes(*w), workspace)) != ADAMW_OK) return rc;
    adamw_matrices_t a = *x, b = *w;
    if (!readable({&a, &b, nullptr}, workspace, st)) return ADAMW_ERR_CUDA;
    return launch_rows(a, b, w->batch, transposed != 0, offsets, *y, st);
}

extern "C" int adamw_expert_outer(const adamw_matrices_t* dy, const adamw_matrices_t* x, const int64_t* offsets,
                                  const adamw_matrices_t* dw, int32_t accumulate, void* workspace, adamw_stream_t stream) {
    int rc = check_outer(dy, x, offsets, dw, accumulate);
    if (rc != ADAMW_OK || dw->rows == 0 || dw->cols == 0) return rc;
    if ((rc = check_workspace(copy_bytes(*dy) + copy_bytes(*x), workspace)) != ADAMW_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    adamw_matrices_t a = *dy, b = *x;
    if (!readable({&a, &b, nullptr}, workspace, st)) return ADAMW_ERR_CUDA;
    return launch_outer(a, b, offsets, *dw, accumulate != 0, st);
}

extern "C" int64_t adamw_expert_backward_workspace(const adamw_matrices_t* dy, const adamw_matrices_t* x, const adamw_matrices_t* w) {
    if (check(dy, true) != ADAMW_OK || check(x, true) != ADAMW_OK || check(w, true) != ADAMW_OK) return 0;
    return copy_bytes(*dy) + copy_bytes(*x) + copy_bytes(*w);
}

extern "C" int adamw_expert_backward(const adamw_matrices_t* dy, const adamw_matrices_t* x, const adamw_matrices_t* w,
                                     int32_t transposed, const int64_t* offsets, const adamw_matrices_t* dx,
                                     const adamw_matrices_t* dw, int32_t dw_transposed, int32_t accumulate, void* workspace,
                                     adamw_stream_t stream) {
    int rc;
    if (!dy || !x || !w || (dw_transposed != 0 && dw_transposed != 1) || (transposed != 0 && transposed != 1)) return ADAMW_ERR_INVALID_ARG;
    const adamw_matrices_t *left = dw_transposed ? x : dy, *right = dw_transposed ? dy : x;
    if (dx && (rc = check_rows(dy, w, !transposed, offsets, dx)) != ADAMW_OK) return rc;
    if (dw && (rc = check_outer(left, right, offsets, dw, accumulate)) != ADAMW_OK) return rc;
    // dx is written before x is read, and w's rows may still be read when dw is written
    if (dx && dw && (dw->batch != w->batch || overlap(*dx, *dw) || overlap(*dx, *x) || overlap(*dw, *w))) return ADAMW_ERR_INVALID_ARG;
    const bool rows = dx && dx->rows > 0 && dx->cols > 0, outer = dw && dw->rows > 0 && dw->cols > 0;
    if (!rows && !outer) return ADAMW_OK;
    const int64_t bytes = copy_bytes(*dy) + (outer ? copy_bytes(*x) : 0) + (rows ? copy_bytes(*w) : 0);
    if ((rc = check_workspace(bytes, workspace)) != ADAMW_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    adamw_matrices_t a = *dy, b = *x, c = *w;
    if (!readable({&a, outer ? &b : nullptr, rows ? &c : nullptr}, workspace, st)) return ADAMW_ERR_CUDA;
    if (rows && (rc = launch_rows(a, c, w->batch, transposed == 0, offsets, *dx, st)) != ADAMW_OK) return rc;
    if (outer) return dw_transposed ? launch_outer(b, a, offsets, *dw, accumulate != 0, st) : launch_outer(a, b, offsets, *dw, accumulate != 0, st);
    return ADAMW_OK;
}
