// token_logprob.cu -- per-token log-probabilities from logits over the
// vocabulary, their gradient, and the policy loss fused with both.
//
// All three are bound by HBM when rows are long or many: a bf16 logit costs
// about five instructions and one exponential (on packed pairs) a pass against
// two bytes.  Few or short rows are bound by latency: a call of one row takes
// 4.7 us.
#include <atomic>

#include "losses_common.cuh"

namespace {

// Threads of a CTA and 16-byte vectors in flight per thread, by kernel.
// Measured with 50272 bf16 logits to a row (us): the forward pass of 8184 rows
// 128 x 8 93.4, 128 x 12 92.5, 128 x 4 94.6, 64 x 8 97.7, 256 x 4 98.4; forward
// and backward of 4092 rows, by the backward's, 128 x 8 165, 256 x 4 165, 128 x
// 4 166, 64 x 8 171; policy of 16376 rows 128 x 8 500, 192 x 4 514, 256 x 4
// 520, 128 x 4 533, 256 x 8 535, 64 x 8 672.
constexpr int kForwardThreads = 128, kForwardUnroll = 8;
constexpr int kBackwardThreads = 128, kBackwardUnroll = 8;
constexpr int kPolicyThreads = 128, kPolicyUnroll = 8;
// Rows of up to this many 16-byte vectors are taken by a warp each, longer ones
// by a CTA or a cluster of them: a short row keeps few loads of a CTA in flight
// between its start and its join.  Measured (bf16, us, warp / CTA), 16384 rows
// of 2048: forward 9.9 / 40.5, with the backward pass 29 / 74, policy 34 / 79;
// of 4096: 22.9 / 42.6, 58 / 85, 53 / 88; of 8192: 41.8 / 47.4, 123 / 121,
// 99 / 99; 64 rows of 4096: 3.0 / 3.8, 5.7 / 6.1, 9.1 / 9.5; of 8192: 4.0 /
// 4.4, 7.7 / 7.2, 10.0 / 10.0.
constexpr int kForwardWarpVecs = 1024, kBackwardWarpVecs = 512, kPolicyWarpVecs = 512;

// The elements of the row outside its vectors, at most one per thread of the
// group: the head's by threads 0.. of the first CTA, the tail's by threads
// 8.. of the last one.  -1: none.
template <int DT>
__device__ __forceinline__ int extra_element(const RowSplit<DT>& sp, int lane, bool first, bool last) {
    if (first && lane < sp.head) return lane;
    if (last && lane >= 8 && lane < 8 + sp.tail) return sp.head + sp.vecs * Elem<DT>::kVec + lane - 8;
    return -1;
}

// Joins the records of a group of threads: a warp, or a cluster of CTAs (one
// or more).  Every thread gets the same record.
template <bool ENT, bool WARP, int THREADS>
__device__ __forceinline__ Online group_join(Online o, float c) {
    o = warp_join<ENT>(o, c);
    if (WARP) {
        __syncwarp();
        return o;
    }
    constexpr int kWarps = THREADS / 32;
    __shared__ Online part[kWarps];
    __shared__ Online whole;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) part[warp] = o;
    __syncthreads();
    o = part[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) join<ENT>(o, part[w], c);
    const uint32_t size = cluster_size();
    if (size > 1) {
        if (threadIdx.x == 0) whole = o;
        cluster_sync();
        for (uint32_t k = 0; k < size; ++k) {
            Online b;
            b.m = load_remote(&whole.m, k);
            b.s = load_remote(&whole.s, k);
            b.t = ENT ? load_remote(&whole.t, k) : 0.0f;
            if (k == 0) o = b; else join<ENT>(o, b, c);
        }
        // no CTA may end, or write its record again, while another reads it
        cluster_sync();
    }
    return o;
}

// The record of a group's row: group_join, and where its largest element is
// extreme, how many are equal to it (a second pass, over such rows only).
// v(i): the i-th of the CTA's n vectors.  xe: the thread's extra element, or
// -inf.
template <int DT, bool ENT, bool WARP, int THREADS, typename Load>
__device__ __forceinline__ Online row_join(Online o, float c, const Load& v, int n, int lane, float xe) {
    using E = Elem<DT>;
    constexpr int width = WARP ? 32 : THREADS;
    o = group_join<ENT, WARP, THREADS>(o, c);
    if (!extreme(o.m, c) || o.s != o.s) return o;   // the whole group
    float count = xe == o.m ? 1.0f : 0.0f;
#pragma unroll 1
    for (int i = lane; i < n; i += width) {
        float x[E::kVec];
        E::unpack(v(i), x);
#pragma unroll
        for (int j = 0; j < E::kVec; ++j) count += x[j] == o.m ? 1.0f : 0.0f;
    }
    if (!WARP) __syncthreads();   // the first join's records have been read
    return group_join<false, WARP, THREADS>({o.m, count, 0.0f}, c);
}

// ---------------------------------------------------------------- forward --

// Log-probability and entropy of one row per group (a warp; or a cluster of
// CTAs, each streaming its share of the row once, with the running maximum
// and sums in registers).  One read of the logits: 8184 rows of 50272 bf16, a
// quarter of them ignored, 94 us, 6.5 TB/s (98 % of this GPU's copy rate).
template <int DT, bool ENT, bool WARP>
__global__ void __launch_bounds__(kForwardThreads)
logprob_kernel(Rows logits, uint32_t rows, int cols, const int64_t* targets, int64_t ignore,
               float scale, float* logp, float* entropy, float* stats) {
    using E = Elem<DT>;
    dependency_trigger();
    dependency_wait();
    const uint32_t size = WARP ? 1 : cluster_size();
    const uint32_t rank = WARP ? 0 : cluster_rank();
    const int lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    constexpr int width = WARP ? 32 : kForwardThreads;
    const uint32_t r = WARP ? blockIdx.x * (kForwardThreads / 32) + threadIdx.x / 32 : blockIdx.x / size;
    if (r >= rows) return;  // whole warps only: the CTA form's grid is exact
    const int64_t t = targets[r];
    const bool writer = lane == 0 && rank == 0;
    if (t == ignore) {
        if (writer) {
            logp[r] = 0.0f;
            if (entropy) entropy[r] = 0.0f;
            if (stats) reinterpret_cast<float2*>(stats)[r] = make_float2(0.0f, kInf);
        }
        return;  // the whole group
    }
    const char* row = logits.at(r);
    const RowSplit<DT> sp(row, cols);
    const float c = scale * kLog2e;
    const uint4* body = reinterpret_cast<const uint4*>(row + int64_t(sp.head) * E::kSize);
    const int first = int(int64_t(sp.vecs) * rank / size);
    const int end = int(int64_t(sp.vecs) * (rank + 1) / size);

    Online o = {-kInf, 0.0f, 0.0f};
    const int extra = extra_element<DT>(sp, lane, rank == 0, rank == size - 1);
    const float xe = extra >= 0 ? E::load(row, extra) : -kInf;
    if (extra >= 0) absorb_one<ENT>(o, xe, c);
    int base = first + lane;
    for (; base + (kForwardUnroll - 1) * width < end; base += kForwardUnroll * width) {
        uint4 v[kForwardUnroll];
#pragma unroll
        for (int u = 0; u < kForwardUnroll; ++u) v[u] = load16(body + base + u * width);
        absorb<DT, ENT>(o, v, c);
    }
    if (base < end) {  // the last few, beside -inf
        uint4 v[kForwardUnroll];
#pragma unroll
        for (int u = 0; u < kForwardUnroll; ++u)
            v[u] = base + u * width < end ? load16(body + base + u * width)
                                          : make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
        absorb<DT, ENT>(o, v, c);
    }
    // for a second pass the row is found again: five registers less over the
    // first, a CTA more on an SM
    auto again = [&](int i) {
        const char* row = logits.at(r);
        return load16(row + int64_t(RowSplit<DT>(row, cols).head) * E::kSize + (int64_t(first) + i) * 16);
    };
    o = row_join<DT, ENT, WARP, kForwardThreads>(o, c, again, end - first, lane, xe);
    if (!writer) return;
    const bool bad = t < 0 || t >= cols;
    RowStats rs = row_stats<ENT>(o);
    if (bad) rs.m = rs.s = rs.log_s = rs.entropy = __int_as_float(0x7fc00000);
    logp[r] = logp_of(rs, bad ? 0.0f : E::load(row, t), scale, c);
    if (entropy) entropy[r] = rs.entropy;
    if (stats) reinterpret_cast<float2*>(stats)[r] = make_float2(rs.m, rs.s);
}

// --------------------------------------------------------------- backward --

// Writes the gradients of the vectors lane, lane + width, .. of n, the first
// of them element `elem` of the row: from v(i), the vector's logits.
template <int DT, bool ENT, int U, typename Load>
__device__ __forceinline__ void grad_vectors(const Gradient& G, const Load& v, int n, int lane, int width,
                                             char* out, bool vector_out, int elem) {
    using E = Elem<DT>;
    if (vector_out && !G.extreme_row) {
        uint4* to = reinterpret_cast<uint4*>(out + int64_t(elem) * E::kSize);
        int i = lane;
        for (; i + (U - 1) * width < n; i += U * width) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = v(i + u * width);
#pragma unroll
            for (int u = 0; u < U; ++u) store16(to + i + u * width, G.of<DT, ENT>(x[u]));
        }
        if (i < n) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U - 1; ++u)
                if (i + u * width < n) x[u] = v(i + u * width);
#pragma unroll
            for (int u = 0; u < U - 1; ++u)
                if (i + u * width < n) store16(to + i + u * width, G.of<DT, ENT>(x[u]));
        }
    } else {  // rows whose addresses differ modulo 16, and rows of extreme logits
        for (int i = lane; i < n; i += width) {
            float x[E::kVec];
            E::unpack(v(i), x);
#pragma unroll
            for (int j = 0; j < E::kVec; ++j) E::store(out, int64_t(elem) + i * E::kVec + j, G.of<ENT>(x[j]));
        }
    }
}

// The target's element, by the thread that wrote it above: its vector is one
// of that thread's, or it is the thread's extra element.
template <int DT, bool ENT>
__device__ __forceinline__ void grad_target(const Gradient& G, char* out, const RowSplit<DT>& sp, int64_t t,
                                            float xt, int first, int end, int lane, int width, int extra) {
    using E = Elem<DT>;
    const int64_t at = t - sp.head, i = at / E::kVec - first;
    const bool in_vectors = at >= 0 && at < int64_t(sp.vecs) * E::kVec;
    const bool mine = in_vectors ? i >= 0 && i < end - first && int(i) % width == lane : t == extra;
    if (mine) E::store(out, t, G.of<ENT>(xt) + G.a);
}

// Zeros in the vectors [first, end) and the extra element of a row.
template <int DT>
__device__ __forceinline__ void zero_row(char* out, bool vector_out, const RowSplit<DT>& sp, int first,
                                         int end, int lane, int width, int extra) {
    using E = Elem<DT>;
    for (int i = first + lane; i < end; i += width) {
        const int elem = sp.head + i * E::kVec;
        if (vector_out) {
            store16(out + int64_t(elem) * E::kSize, make_uint4(0, 0, 0, 0));
        } else {
            for (int j = 0; j < E::kVec; ++j) E::store(out, elem + j, 0.0f);
        }
    }
    if (extra >= 0) E::store(out, extra, 0.0f);
}

// Elementwise from the row's maximum and sum, one CTA per piece of a row (or a
// warp per row).  zeros: a row whose gradients are 0 is not used (it may hold
// anything) and gets 0.  4092 rows of 50272 bf16, a quarter of them ignored, after
// their forward pass: 109 us, 6.6 TB/s over one read and one write.
template <int DT, bool ENT, bool WARP>
__global__ void __launch_bounds__(kBackwardThreads)
logprob_backward_kernel(Rows logits, Rows grad, uint32_t rows, uint32_t pieces, int cols,
                        const int64_t* targets, float scale, const float* stats, const float* entropy,
                        const float* d_logp, const float* d_entropy, bool zeros) {
    using E = Elem<DT>;
    dependency_trigger();
    dependency_wait();
    const int lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    constexpr int width = WARP ? 32 : kBackwardThreads;
    // the last rows first: a forward pass just before left them in L2
    const uint32_t back = WARP ? blockIdx.x * (kBackwardThreads / 32) + threadIdx.x / 32 : blockIdx.x / pieces;
    const uint32_t piece = WARP ? 0 : blockIdx.x - back * pieces;
    if (back >= rows) return;
    const uint32_t r = rows - 1 - back;
    const char* row = logits.at(r);
    char* out = grad.at(r);
    const RowSplit<DT> sp(row, cols);
    const bool vector_out = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int first = int(int64_t(sp.vecs) * piece / pieces);
    const int end = int(int64_t(sp.vecs) * (piece + 1) / pieces);
    const int extra = extra_element<DT>(sp, lane, piece == 0, piece == pieces - 1);

    const float2 st = reinterpret_cast<const float2*>(stats)[r];
    const int64_t t = targets[r];
    const float a = scale * d_logp[r];
    const float b = ENT ? scale * d_entropy[r] : 0.0f;
    const float H = ENT ? entropy[r] : 0.0f;
    // ignored, without a distribution, or of a token that does not count
    if (st.y == kInf || (zeros && a == 0.0f && b == 0.0f)) {
        zero_row<DT>(out, vector_out, sp, first, end, lane, width, extra);
        return;
    }
    const float xt = t >= 0 && t < cols ? E::load(row, t) : 0.0f;
    const Gradient G(st.x, st.y, ENT ? logf(st.y) : 0.0f, scale * kLog2e, a, b, H);
    const uint4* body = reinterpret_cast<const uint4*>(row + int64_t(sp.head) * E::kSize) + first;
    const float xe = extra >= 0 ? E::load(row, extra) : 0.0f;
    grad_vectors<DT, ENT, kBackwardUnroll>(G, [body](int i) { return load16(body + i); }, end - first, lane, width, out,
                                   vector_out, sp.head + first * E::kVec);
    if (extra >= 0) E::store(out, extra, G.of<ENT>(xe));
    grad_target<DT, ENT>(G, out, sp, t, xt, first, end, lane, width, extra);
}

// ------------------------------------------------------ fused policy loss --

struct PolicyRows {
    const int64_t* targets;
    int64_t ignore;
    const float *old_logp, *ref_logp, *advantages;
    const Counts* counts;
    float *logp, *entropy;
};

__device__ __forceinline__ void copy_async16(uint4* smem, const uint4* global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// Groups of kPolicyUnroll vectors per thread that are on their way at a time.
constexpr int kDepth = 4;

// The policy loss of one token per group, from its row of logits to their
// gradient: the row (each CTA's share of it) is copied to shared memory with
// the maximum and sums taken as it arrives, the group joins them, every
// thread works out the token's loss, and the gradient is written from the
// copy: one read and one write of HBM.  A thread reads only the vectors that
// it copied itself, so the copies need no barrier.  With the count before and
// the statistics after it, 16376 rows of 50272 bf16 (a quarter of them ignored,
// with the entropy) take 502 us, 5.7 TB/s; without the entropy and with none
// ignored 16384 rows take 549 us, 6.0 TB/s, where a 16-byte copy kernel reaches
// 6.26.  Two rows are on an SM, eight warps, which issue in 46 % of the cycles
// (thirds of rows in registers, three rows to an SM, gave 0 to 2 %).
template <int DT, bool ENT, bool WARP>
__global__ void __launch_bounds__(kPolicyThreads)
policy_rows_kernel(Rows logits, Rows grad, Tokens tokens, int cols, float scale, Policy P, PolicyRows a) {
    using E = Elem<DT>;
    extern __shared__ uint4 slices[];
    dependency_trigger();
    dependency_wait();
    const uint32_t size = WARP ? 1 : cluster_size();
    const uint32_t rank = WARP ? 0 : cluster_rank();
    const int lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    constexpr int width = WARP ? 32 : kPolicyThreads;
    const uint32_t r = WARP ? blockIdx.x * (kPolicyThreads / 32) + threadIdx.x / 32 : blockIdx.x / size;
    if (r >= tokens.n) return;
    const char* row = logits.at(r);
    char* out = grad.at(r);
    const RowSplit<DT> sp(row, cols);
    const bool vector_out = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int first = int(int64_t(sp.vecs) * rank / size);
    const int end = int(int64_t(sp.vecs) * (rank + 1) / size);
    const int extra = extra_element<DT>(sp, lane, rank == 0, rank == size - 1);
    const bool writer = lane == 0 && rank == 0;

    const int64_t t = a.targets[r];
    if (t == a.ignore) {
        zero_row<DT>(out, vector_out, sp, first, end, lane, width, extra);
        if (writer) {
            a.logp[r] = 0.0f;
            if (a.entropy) a.entropy[r] = 0.0f;
        }
        return;  // the whole group
    }
    uint4* slice = slices + (WARP ? (threadIdx.x / 32) * (cols / E::kVec) : 0);
    const uint4* body = reinterpret_cast<const uint4*>(row + int64_t(sp.head) * E::kSize) + first;
    const int n = end - first;
    int asked = lane;
    auto ask = [&] {
#pragma unroll
        for (int u = 0; u < kPolicyUnroll; ++u)
            if (asked + u * width < n) copy_async16(slice + asked + u * width, body + asked + u * width);
        asked += kPolicyUnroll * width;
        copy_commit();
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) ask();

    const float c = scale * kLog2e;
    const bool bad = t < 0 || t >= cols;
    const float xt = bad ? 0.0f : E::load(row, t);
    const float xe = extra >= 0 ? E::load(row, extra) : -kInf;
    const float old = a.old_logp[r];
    const float ref = a.ref_logp ? a.ref_logp[r] : 0.0f;
    const int32_t seq = tokens.sequence(r);
    const float A = seq < 0 ? 0.0f : a.advantages[P.per_token ? r : uint32_t(seq)];
    const float w = seq < 0 ? 0.0f
                            : token_weight(P.reduce, P.inv_divisor, a.counts->tokens, a.counts->filled,
                                           a.counts->sequence[seq]) * P.grad_scale;

    Online o = {-kInf, 0.0f, 0.0f};
    if (extra >= 0) absorb_one<ENT>(o, xe, c);
    for (int base = lane; base < n; base += kPolicyUnroll * width) {
        copy_wait<kDepth - 1>();
        if (base + (kPolicyUnroll - 1) * width < n) {
            uint4 v[kPolicyUnroll];
#pragma unroll
            for (int u = 0; u < kPolicyUnroll; ++u) v[u] = slice[base + u * width];
            absorb<DT, ENT>(o, v, c);
        } else {
            for (int i = base; i < n; i += width) {
                const uint4 v[1] = {slice[i]};
                absorb<DT, ENT>(o, v, c);
            }
        }
        ask();
    }
    o = row_join<DT, ENT, WARP, kPolicyThreads>(o, c, [slice](int i) { return slice[i]; }, n, lane, xe);

    RowStats rs = row_stats<ENT>(o);
    if (bad) rs.m = rs.s = rs.log_s = rs.entropy = __int_as_float(0x7fc00000);
    const float lp = logp_of(rs, xt, scale, c);
    if (writer) {
        a.logp[r] = lp;
        if (a.entropy) a.entropy[r] = rs.entropy;
    }
    const PolicyToken k = policy_token(P, lp, old, a.ref_logp != nullptr, ref, A);
    if (rs.s == kInf || seq < 0) {
        zero_row<DT>(out, vector_out, sp, first, end, lane, width, extra);
        return;
    }
    const Gradient G(rs.m, rs.s, rs.log_s, c, scale * w * k.grad, ENT ? -scale * w * P.entropy_coef : 0.0f,
                     rs.entropy);
    grad_vectors<DT, ENT, kPolicyUnroll>(G, [slice](int i) { return slice[i]; }, n, lane, width, out, vector_out,
                                   sp.head + first * E::kVec);
    if (extra >= 0) E::store(out, extra, G.of<ENT>(xe));
    grad_target<DT, ENT>(G, out, sp, t, xt, first, end, lane, width, extra);
}

// ------------------------------------------------------------------- host --

// Fewest CTAs that keep the GPU busy: where there are fewer rows, each is
// split over a cluster: one for each of the 152 SMs of a GB300, for which this
// library is built.  Measured (50272 elements, us, split / not): forward
// of 1 row 4.7 / 5.8, of 32 5.3 / 6.0, of 76 5.7 / 6.0, of 152 6.1 / 6.3;
// policy of 1 row 11.6 / 13.7, of 32 12.0 / 13.7, of 76 13.3 / 13.9, of 152
// 15.5 / 15.3.  Splitting further, up to 608 CTAs, costs 1 to 2 us.
constexpr int64_t kBusyCtas = 152;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxSmem = 200 * 1024;    // a CTA's share of a row, at most
constexpr int64_t kWantSmem = 108 * 1024;   // two CTAs to an SM

int vec_of(int32_t dt) { return dt == ADAMW_DTYPE_FP32 ? 4 : 8; }

bool same_rows(const adamw_rows_t* a, const adamw_rows_t* b) {
    return a->data == b->data && a->inner == b->inner &&
           (a->inner == 1 || a->row_stride == b->row_stride) &&
           (a->rows == a->inner || a->outer_stride == b->outer_stride);
}

// Elements from the first of `data` to one past the last.
int64_t extent(const adamw_rows_t* m) {
    if (m->rows == 0) return 0;
    return (m->rows / m->inner - 1) * m->outer_stride + (m->inner - 1) * m->row_stride + m->cols;
}

int check_rows(const adamw_rows_t* m, bool written) {
    if (!m || m->rows < 0 || m->cols < 0 || m->inner < 1 || m->outer_stride < 0 || m->row_stride < 0)
        return ADAMW_ERR_INVALID_ARG;
    const int size = dtype_size(m->dtype);
    if (size == 0) return ADAMW_ERR_INVALID_ARG;
    if (m->rows == 0) return ADAMW_OK;
    if (!m->data || m->cols < 1 || m->rows % m->inner != 0) return ADAMW_ERR_INVALID_ARG;
    if (m->rows > kMaxCount) return ADAMW_ERR_TOO_LARGE;
    // offsets stay far inside 64 bits
    constexpr int64_t kMaxStride = int64_t(1) << 40;
    if (m->outer_stride > kMaxStride || m->row_stride > kMaxStride) return ADAMW_ERR_TOO_LARGE;
    const int64_t outer = m->rows / m->inner;
    if ((outer > 1 && m->outer_stride > (int64_t(1) << 60) / outer) ||
        (m->inner > 1 && m->row_stride > (int64_t(1) << 60) / m->inner))
        return ADAMW_ERR_TOO_LARGE;
    if (!aligned(m->data, uintptr_t(size))) return ADAMW_ERR_MISALIGNED;
    if (written) {
        // rows apart from one another, the smaller stride's run inside the larger
        const bool in = m->inner > 1, out = outer > 1;
        const int64_t small = in && out ? (m->row_stride < m->outer_stride ? m->row_stride : m->outer_stride)
                              : in ? m->row_stride : m->outer_stride;
        if ((in || out) && small < m->cols) return ADAMW_ERR_INVALID_ARG;
        if (in && out) {
            const bool rows_inside = m->row_stride <= m->outer_stride;
            const int64_t run = rows_inside ? (m->inner - 1) * m->row_stride : (outer - 1) * m->outer_stride;
            if ((rows_inside ? m->outer_stride : m->row_stride) < run + m->cols) return ADAMW_ERR_INVALID_ARG;
        }
    }
    return ADAMW_OK;
}

int check_gradient(const adamw_rows_t* x, const adamw_rows_t* d) {
    int rc = check_rows(d, true);
    if (rc != ADAMW_OK) return rc;
    if (d->rows != x->rows || d->cols != x->cols || d->dtype != x->dtype) return ADAMW_ERR_INVALID_ARG;
    if (x->rows == 0 || same_rows(x, d)) return ADAMW_OK;
    const uintptr_t size = uintptr_t(dtype_size(x->dtype));
    const uintptr_t a = reinterpret_cast<uintptr_t>(x->data), b = reinterpret_cast<uintptr_t>(d->data);
    const bool apart = a + uintptr_t(extent(x)) * size <= b || b + uintptr_t(extent(d)) * size <= a;
    return apart ? ADAMW_OK : ADAMW_ERR_INVALID_ARG;
}

Rows rows_of(const adamw_rows_t* m) {
    Rows r;
    const int64_t size = dtype_size(m->dtype);
    r.data = static_cast<char*>(m->data);
    r.outer = m->outer_stride * size;
    r.row = m->row_stride * size;
    r.inner = uint32_t(m->inner);
    return r;
}

bool good_scale(float s) { return s > 0.0f && std::isfinite(s * kLog2e); }

// CTAs per row: one where there are rows enough to keep the GPU busy, else up
// to eight, each with at least two turns of its threads' vectors.
int cluster_for(int64_t rows, int64_t vecs, int threads, int at_least) {
    int c = at_least;
    while (c < kMaxCluster && rows * c < kBusyCtas && vecs >= int64_t(2) * c * 2 * threads) c *= 2;
    return c;
}

// The grid of the warp form: a row to each warp.
uint32_t warp_grid(uint32_t rows, int threads) { return (rows + uint32_t(threads / 32) - 1) / uint32_t(threads / 32); }

uint32_t grid_of(int64_t groups) { return groups > 0 && groups <= kMaxCount ? uint32_t(groups) : 0; }

template <int DT>
cudaError_t forward(const adamw_rows_t* x, const int64_t* targets, int64_t ignore, float scale,
                    float* logp, float* entropy, float* stats, cudaStream_t st) {
    const Rows rows = rows_of(x);
    const uint32_t n = uint32_t(x->rows);
    if (x->cols / Elem<DT>::kVec <= kForwardWarpVecs) {
        auto k = entropy ? logprob_kernel<DT, true, true> : logprob_kernel<DT, false, true>;
        return launch(k, warp_grid(n, kForwardThreads), kForwardThreads, 1, 0, st, rows, n, x->cols, targets, ignore,
                      scale, logp, entropy, stats);
    }
    const int c = cluster_for(x->rows, x->cols / Elem<DT>::kVec, kForwardThreads, 1);
    auto k = entropy ? logprob_kernel<DT, true, false> : logprob_kernel<DT, false, false>;
    const uint32_t grid = grid_of(x->rows * c);
    if (!grid) return cudaErrorInvalidConfiguration;
    return launch(k, grid, kForwardThreads, c, 0, st, rows, n, x->cols, targets, ignore, scale, logp, entropy, stats);
}

template <int DT>
cudaError_t backward(const adamw_rows_t* x, const int64_t* targets, float scale, const float* stats,
                     const float* entropy, const float* d_logp, const float* d_entropy, bool zeros,
                     const adamw_rows_t* dx, cudaStream_t st) {
    const Rows in = rows_of(x), out = rows_of(dx);
    const uint32_t n = uint32_t(x->rows);
    if (x->cols / Elem<DT>::kVec <= kBackwardWarpVecs) {
        auto k = d_entropy ? logprob_backward_kernel<DT, true, true> : logprob_backward_kernel<DT, false, true>;
        return launch(k, warp_grid(n, kBackwardThreads), kBackwardThreads, 1, 0, st, in, out, n, 1u, x->cols, targets,
                      scale, stats, entropy, d_logp, d_entropy, zeros);
    }
    // two turns of its threads' vectors to a piece
    const int64_t per = 2 * int64_t(kBackwardThreads) * kBackwardUnroll * Elem<DT>::kVec;
    const uint32_t pieces = uint32_t((x->cols + per - 1) / per);
    auto k = d_entropy ? logprob_backward_kernel<DT, true, false> : logprob_backward_kernel<DT, false, false>;
    const uint32_t grid = grid_of(x->rows * pieces);
    if (!grid) return cudaErrorInvalidConfiguration;
    return launch(k, grid, kBackwardThreads, 1, 0, st, in, out, n, pieces, x->cols, targets, scale, stats, entropy,
                  d_logp, d_entropy, zeros);
}

int launch_backward(const adamw_rows_t* x, const int64_t* targets, float scale, const float* stats,
                    const float* entropy, const float* d_logp, const float* d_entropy, bool zeros,
                    const adamw_rows_t* dx, cudaStream_t st) {
    cudaError_t e;
    switch (x->dtype) {
        case ADAMW_DTYPE_BF16: e = backward<ADAMW_DTYPE_BF16>(x, targets, scale, stats, entropy, d_logp, d_entropy, zeros, dx, st); break;
        case ADAMW_DTYPE_FP16: e = backward<ADAMW_DTYPE_FP16>(x, targets, scale, stats, entropy, d_logp, d_entropy, zeros, dx, st); break;
        default: e = backward<ADAMW_DTYPE_FP32>(x, targets, scale, stats, entropy, d_logp, d_entropy, zeros, dx, st); break;
    }
    return launched(e, "token_logprob_backward launch") ? ADAMW_OK : ADAMW_ERR_CUDA;
}

// Allows a kernel its dynamic shared memory, once per device.
cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// A row's vectors in shared memory fit a cluster.
bool fits_cluster(const adamw_rows_t* x) {
    return int64_t(x->cols / vec_of(x->dtype)) * 16 <= int64_t(kMaxCluster) * (kMaxSmem - 16);
}

template <int DT, bool ENT>
cudaError_t policy_rows(const adamw_rows_t* x, const adamw_rows_t* dx, const Tokens& tokens, float scale,
                        const Policy& P, const PolicyRows& a, cudaStream_t st) {
    const Rows in = rows_of(x), out = rows_of(dx);
    const int64_t vecs = x->cols / Elem<DT>::kVec;
    if (vecs <= kPolicyWarpVecs)   // at most 8 KB to a warp
        return launch(policy_rows_kernel<DT, ENT, true>, warp_grid(tokens.n, kPolicyThreads), kPolicyThreads, 1,
                      size_t(vecs) * 16 * (kPolicyThreads / 32), st, in, out, tokens, x->cols, scale, P, a);
    auto k = policy_rows_kernel<DT, ENT, false>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), done);
    if (e != cudaSuccess) return e;
    int c = 1;
    while (c < kMaxCluster && (vecs + c - 1) / c * 16 > kWantSmem) c *= 2;
    c = cluster_for(x->rows, vecs, kPolicyThreads, c);
    const uint32_t grid = grid_of(x->rows * c);
    if (!grid) return cudaErrorInvalidConfiguration;
    return launch(k, grid, kPolicyThreads, c, size_t((vecs + c - 1) / c) * 16, st, in, out, tokens, x->cols,
                  scale, P, a);
}

template <int DT>
cudaError_t policy_rows(const adamw_rows_t* x, const adamw_rows_t* dx, const Tokens& tokens, float scale,
                        const Policy& P, const PolicyRows& a, cudaStream_t st) {
    return a.entropy ? policy_rows<DT, true>(x, dx, tokens, scale, P, a, st)
                     : policy_rows<DT, false>(x, dx, tokens, scale, P, a, st);
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

extern "C" int adamw_token_logprob(const adamw_rows_t* logits, const int64_t* targets,
                                   int64_t ignore_index, float scale, float* logp, float* entropy,
                                   float* stats, adamw_stream_t stream) {
    const int rc = check_rows(logits, false);
    if (rc != ADAMW_OK) return rc;
    if (!good_scale(scale)) return ADAMW_ERR_INVALID_ARG;
    if (logits->rows == 0) return ADAMW_OK;
    if (!targets || !logp) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(targets, 8) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(stats, 8))
        return ADAMW_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (logits->dtype) {
        case ADAMW_DTYPE_BF16: e = forward<ADAMW_DTYPE_BF16>(logits, targets, ignore_index, scale, logp, entropy, stats, st); break;
        case ADAMW_DTYPE_FP16: e = forward<ADAMW_DTYPE_FP16>(logits, targets, ignore_index, scale, logp, entropy, stats, st); break;
        default: e = forward<ADAMW_DTYPE_FP32>(logits, targets, ignore_index, scale, logp, entropy, stats, st); break;
    }
    return launched(e, "token_logprob launch") ? ADAMW_OK : ADAMW_ERR_CUDA;
}

extern "C" int adamw_token_logprob_backward(const adamw_rows_t* logits, const int64_t* targets,
                                            int64_t ignore_index, float scale, const float* stats,
                                            const float* entropy, const float* d_logp,
                                            const float* d_entropy, const adamw_rows_t* d_logits,
                                            adamw_stream_t stream) {
    (void)ignore_index;  // the forward call marked those rows in stats
    int rc = check_rows(logits, false);
    if (rc != ADAMW_OK) return rc;
    if (!d_logits) return ADAMW_ERR_INVALID_ARG;
    rc = check_gradient(logits, d_logits);
    if (rc != ADAMW_OK) return rc;
    if (!good_scale(scale)) return ADAMW_ERR_INVALID_ARG;
    if (logits->rows == 0) return ADAMW_OK;
    if (!targets || !stats || !d_logp || (d_entropy && !entropy)) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(targets, 8) || !aligned(stats, 8) || !aligned(d_logp, 4) || !aligned(d_entropy, 4) ||
        !aligned(entropy, 4))
        return ADAMW_ERR_MISALIGNED;
    return launch_backward(logits, targets, scale, stats, entropy, d_logp, d_entropy, false, d_logits,
                           reinterpret_cast<cudaStream_t>(stream));
}

// The workspace: the policy loss's, then (used for rows too long for a
// cluster) the forward pass's stats and the gradients of logp and entropy.
extern "C" int64_t adamw_policy_logits_workspace(int64_t n, int64_t sequences) {
    const int64_t base = adamw_policy_workspace(n, sequences);
    return base == 0 ? 0 : round16(base) + round16(8 * n) + 2 * round16(4 * n);
}

extern "C" int adamw_policy_loss_logits(const adamw_rows_t* logits, const int64_t* targets,
                                        int64_t ignore_index, float scale, const adamw_tokens_t* tokens,
                                        const adamw_policy_t* policy, const float* old_logp,
                                        const float* ref_logp, const float* advantages, float* stats,
                                        int64_t* counts, float* logp, float* entropy,
                                        const adamw_rows_t* d_logits, void* workspace,
                                        adamw_stream_t stream) {
    int rc = check_rows(logits, false);
    if (rc != ADAMW_OK) return rc;
    if (!d_logits) return ADAMW_ERR_INVALID_ARG;
    rc = check_gradient(logits, d_logits);
    if (rc != ADAMW_OK) return rc;
    rc = adamw::check_tokens(tokens);
    if (rc != ADAMW_OK) return rc;
    rc = adamw::check_policy(policy);
    if (rc != ADAMW_OK) return rc;
    if (!good_scale(scale) || tokens->mask || tokens->n != logits->rows) return ADAMW_ERR_INVALID_ARG;
    if (!stats || !counts || !workspace || (policy->entropy_coef != 0.0f && !entropy) ||
        (policy->kl_coef != 0.0f && !ref_logp))
        return ADAMW_ERR_INVALID_ARG;
    if (tokens->n > 0 && (!targets || !old_logp || !advantages || !logp)) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(targets, 8) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(advantages, 4) ||
        !aligned(stats, 4) || !aligned(counts, 8) || !aligned(logp, 4) || !aligned(entropy, 4) ||
        !aligned(workspace, 16))
        return ADAMW_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    rc = adamw::launch_counts(tokens, targets, ignore_index, workspace, st);
    if (rc != ADAMW_OK) return rc;
    if (tokens->n == 0 || fits_cluster(logits)) {
        if (tokens->n > 0) {
            const Tokens t = tokens_of(tokens, targets, ignore_index);
            const Policy P = policy_of(policy);
            const PolicyRows a = {targets, ignore_index, old_logp, ref_logp, advantages,
                                  static_cast<const Counts*>(workspace), logp, entropy};
            cudaError_t e;
            switch (logits->dtype) {
                case ADAMW_DTYPE_BF16: e = policy_rows<ADAMW_DTYPE_BF16>(logits, d_logits, t, scale, P, a, st); break;
                case ADAMW_DTYPE_FP16: e = policy_rows<ADAMW_DTYPE_FP16>(logits, d_logits, t, scale, P, a, st); break;
                default: e = policy_rows<ADAMW_DTYPE_FP32>(logits, d_logits, t, scale, P, a, st); break;
            }
            if (!launched(e, "policy_loss_logits launch")) return ADAMW_ERR_CUDA;
        }
        return adamw::launch_policy(tokens, policy, targets, ignore_index, true, logp, old_logp, ref_logp,
                                    advantages, entropy, stats, counts, nullptr, nullptr, workspace, st);
    }
    char* w = static_cast<char*>(workspace) + round16(adamw_policy_workspace(tokens->n, tokens->sequences));
    float* row_stats = reinterpret_cast<float*>(w);
    float* d_logp = reinterpret_cast<float*>(w + round16(8 * tokens->n));
    float* d_entropy = entropy ? reinterpret_cast<float*>(w + round16(8 * tokens->n) + round16(4 * tokens->n)) : nullptr;
    rc = adamw_token_logprob(logits, targets, ignore_index, scale, logp, entropy, row_stats, stream);
    if (rc != ADAMW_OK) return rc;
    rc = adamw::launch_policy(tokens, policy, targets, ignore_index, true, logp, old_logp, ref_logp, advantages,
                              entropy, stats, counts, d_logp, d_entropy, workspace, st);
    if (rc != ADAMW_OK) return rc;
    return launch_backward(logits, targets, scale, row_stats, entropy, d_logp, d_entropy, true, d_logits, st);
}
