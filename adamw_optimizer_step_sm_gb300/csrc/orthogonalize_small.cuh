// orthogonalize_small.cuh -- the whole iteration of small matrices in one
// kernel: a cluster of up to eight CTAs has a matrix of at most 128 x 1024 (or
// 1024 x 128), 128 of the long side each, and takes all steps on chip.
// Included by orthogonalize.cu, whose products take 17 launches for a matrix
// of any size, each a few microseconds whatever it computes.
//
// X stays in registers, in fp32; shared memory holds what the tensor cores
// read, in fp16 at 2^12 times its value as in the large form: X's part, G and Q.
// Q X takes X and Q as two fp16 each (three products: 22 against 17 us for 64 x 128):
// in small matrices the roundings of few numbers do not average out (figures in
// orthogonalize.cu). The sum G = X X^T over the cluster goes through distributed
// shared memory, in fp32: each CTA adds up its share of G over all parts, in their
// order, and hands the sums to all.
//
// Bound by latency: a step is three products one after the other, each half a
// microsecond of tensor cores and as much between their operands and results in
// shared memory; a cluster adds two barriers (1.2 us a step) and the exchange (0.3 for a
// side of 32, 2 for one of 128). One 64 x 128 takes 20 us in a row of them, 64 x 1024 29,
// 128 x 1024 37, the Muon step of twelve of 128 x 128 to 512 61.
#pragma once

namespace {

constexpr int kSmallThreads = 256;
constexpr int kSmallSide = 128, kSmallMost = 8;   // largest side, CTAs of a cluster
constexpr uint32_t kPlane = 128 * 128;            // 64 columns of 128 rows of fp16
// Two planes each for X, what its fp16 leaves, G, Q, what Q's fp16 leaves (a cluster's
// parts of G, in fp32, have the place of both), and what G's leaves.
constexpr uint32_t kSmallBytes = 1024 + 12 * kPlane;

template <bool MUON>
struct SmallParams {
    CopyParams<MUON> in;              // shapes, source, norms of a plan
    int32_t first_cluster[kMaxShapes];
    float rate[kMaxShapes];
    float coefs[32][3];
    int32_t steps, pretend;
    Batch dst;
};

struct SmallControl {
    uint64_t done;
    uint32_t tmem;
    int32_t failed;
    double part[kSmallThreads / 32], sum;
};

// 16-byte unit j (eight columns) of row r in a plane, as the tensor cores read it.
__device__ __forceinline__ uint32_t unit_at(int r, int j) { return uint32_t(r * 128 + ((j ^ (r & 7)) << 4)); }

// What fp16 leaves of eight values, in fp16.
__device__ __forceinline__ uint4 left_of(const float* v) {
    float h[8];
    Fp16::unpack(Fp16::pack(v), h);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = v[e] - h[e];
    return Fp16::pack(h);
}

// A cluster's sums of G go by blocks of 8 x 8, those on and below the diagonal that the
// matrix has, each in one piece: what eight lanes read or write of another CTA is one row
// of 128 bytes.  Reads bound this: rows of all of G in fp32 took 41.4 us for 128 x 1024 and 38.1
// for 64 x 1024; of the half in blocks by 16 bytes 54.2 and 34.6; this 37.0 and 28.5.
constexpr int kBlocksOfG = 16 * 17 / 2;
constexpr uint32_t kSums = kBlocksOfG * 256, kSumsLow = kSums + kBlocksOfG * 128;   // behind the parts, in fp32
static_assert(kSumsLow + (kFineSide / 8) * (kFineSide / 8 + 1) / 2 * 128 <= 4 * kPlane, "in the place of Q");

__device__ __forceinline__ int block_of(int down, int across) { return down * (down + 1) / 2 + across; }

// 16 bytes to the same place of all CTAs of the cluster.
template <int CTAS>
__device__ __forceinline__ void hand_out(const unsigned char* at, uint4 g) {
#pragma unroll
    for (int o = 0; o < CTAS; ++o)
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(in_cta(smem_addr(at), uint32_t(o))), "r"(g.x), "r"(g.y),
                     "r"(g.z), "r"(g.w) : "memory");
}

// This CTA's share of the blocks, added up over the cluster's parts in their order, and
// handed to all in fp16, with what that leaves where `fine`.
template <int CTAS, bool FINE>
__device__ __forceinline__ void add_up(unsigned char* parts, bool fine, int blocks, uint32_t rank) {
    const int e = int(threadIdx.x) % 8;
#pragma unroll 1
    for (int t = int(rank) + CTAS * (int(threadIdx.x) / 8); t < blocks; t += CTAS * kSmallThreads / 8) {
        float4 v[CTAS][2];
#pragma unroll
        for (int o = 0; o < CTAS; ++o)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float4& w = v[o][half];
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                             : "r"(in_cta(smem_addr(parts + t * 256 + half * 128 + e * 16), uint32_t(o))) : "memory");
            }
        float sum[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float4 w = v[0][half];
#pragma unroll
            for (int o = 1; o < CTAS; ++o) w = make_float4(w.x + v[o][half].x, w.y + v[o][half].y, w.z + v[o][half].z, w.w + v[o][half].w);
            sum[half * 4] = w.x, sum[half * 4 + 1] = w.y, sum[half * 4 + 2] = w.z, sum[half * 4 + 3] = w.w;
        }
        hand_out<CTAS>(parts + kSums + t * 128 + e * 16, Fp16::pack(sum));
        if (FINE && fine) hand_out<CTAS>(parts + kSumsLow + t * 128 + e * 16, left_of(sum));
    }
}

// The sums as the tensor cores read them: each block and its transpose.  A warp has two of
// the n rows of blocks, n even, together as many as any other's, four blocks at a time.
__device__ __forceinline__ void lay_out(const unsigned char* sums, unsigned char* g, int n) {
    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32, e = lane % 8;
    if (warp >= n / 2) return;
#pragma unroll 1
    for (int i = 0; i <= n; i += 4) {
        const int q = i + lane / 8 <= n ? i + lane / 8 : n;   // the last one again: the same numbers to the same place
        const int down = q <= warp ? warp : n - 1 - warp, across = q <= warp ? q : q - warp - 1;
        const uint32_t from = smem_addr(sums + block_of(down, across) * 128 + e * 16);
        uint32_t a, b, c, d;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(from) : "memory");
        const uint32_t to = smem_addr(g + across / 8 * kPlane + unit_at(down * 8 + e, across % 8));
        const uint32_t turned = smem_addr(g + down / 8 * kPlane + unit_at(across * 8 + e, down % 8));
        asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
        __syncwarp();   // a block on the diagonal is written twice
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(turned), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
    }
}

// FINE: some shape is (as a flag at run time alone: 64 x 128 8 % slower).
template <bool MUON, int DT, bool FINE>
__global__ void __launch_bounds__(kSmallThreads, 1) small_kernel(const __grid_constant__ SmallParams<MUON> p) {
    extern __shared__ unsigned char raw[];
    __shared__ SmallControl ctl;
    unsigned char* base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    unsigned char *xs = base, *xl = base + 2 * kPlane, *gs = base + 4 * kPlane, *qs = base + 6 * kPlane, *ql = base + 8 * kPlane, *gl = base + 10 * kPlane;
    unsigned char* parts = qs;   // of G, in a cluster

    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int r = warp % 4 * 32 + lane, h = warp / 4;   // the thread's row, and its 64 columns
    const uint32_t bar = smem_addr(&ctl.done);
    if (threadIdx.x == 0) {
        barrier_init(bar, 1);
        ctl.failed = p.pretend ? Waiter::kPretend : 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc<1>(smem_addr(&ctl.tmem), 128);
    int k = 0;
    const int cluster = int(blockIdx.x / ctas);
    while (k + 1 < p.in.n && p.first_cluster[k + 1] <= cluster) ++k;
    const CopyShape& c = p.in.shapes[k];
    const int matrix = cluster - p.first_cluster[k];
    const int rows = c.s.rows, cols = c.s.cols, side = c.s.side;
    const bool wide = rows <= cols, fine = FINE && c.s.fine;
    const int at = int(rank) * 128, length = wide ? cols : rows;
    const int mine = length - at < 0 ? 0 : length - at < 128 ? length - at : 128;   // of the long side
    tmem_before();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = *static_cast<volatile uint32_t*>(&ctl.tmem) + (uint32_t(warp % 4 * 32) << 16) + uint32_t(h * 64);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool skip = MUON && *p.in.nonfinite != 0;

    // ---- X, unscaled, and its norm
    const Source<MUON, DT> src(p.in, c, matrix);
    float x[64];
    const int valid = r < side ? (mine - h * 64 < 64 ? mine - h * 64 : 64) : 0;   // of the thread's values
    // all loads of a batch before its first store, which they would wait for
    if (wide) {
        Raw w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j * 8 < valid) w[j] = src.load(r, at + h * 64 + j * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float u[8], m[8];
            if (j * 8 < valid) {
                src.value(w[j], u, m);
                if (MUON && !skip) src.put(r, at + h * 64 + j * 8, m);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j * 8 + e] = j * 8 + e < valid ? u[e] : 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 64; i += 32) {
            float m[MUON ? 32 : 1];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[i + e] = i + e < valid ? src.one(at + h * 64 + i + e, r, m + (MUON ? e : 0)) : 0.0f;
            if (MUON && !skip) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (i + e < valid) src.put_one(at + h * 64 + i + e, r, m[MUON ? e : 0]);
            }
        }
    }
    double sum = 0.0;
    if (MUON) {
        for (int i = 0; i < c.pieces; ++i) sum += p.in.sums[c.first_sum + matrix * c.pieces + i];
    } else {
        Sum2 total = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s = 0.0f, any = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s = fmaf(x[j * 8 + e], x[j * 8 + e], s);
                any = any == 0.0f ? x[j * 8 + e] : any;
            }
            if (s >= 0x1p-100f && s <= 0x1p100f) {
                total.add(s);
            } else if (any != 0.0f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += double(x[j * 8 + e]) * double(x[j * 8 + e]);
            }
        }
        sum += double(total.hi) + double(total.lo);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) ctl.part[warp] = sum;
        __syncthreads();
        sum = 0.0;
        for (int i = 0; i < kSmallThreads / 32; ++i) sum += ctl.part[i];
        if (ctas > 1) {
            if (threadIdx.x == 0) ctl.sum = sum;
            cluster_sync();
            sum = 0.0;
            for (uint32_t i = 0; i < ctas; ++i) {
                double v;
                asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(in_cta(smem_addr(&ctl.sum), i)) : "memory");
                sum += v;
            }
        }
    }
    const Scale scale = scale_of(sum, p.in.eps);
    scale(x);

    // ---- the steps
    uint32_t turn = 0;
    const Waiter wait = {&ctl.failed};
    const uint32_t xa = smem_addr(xs), xla = smem_addr(xl), ga = smem_addr(gs), qa = smem_addr(qs), qla = smem_addr(ql), gla = smem_addr(gl), out = *static_cast<volatile uint32_t*>(&ctl.tmem);
    // what is there of k; all 128 rows and columns are computed, zeros beyond the matrix
    const int side16 = (side + 15) / 16 * 16, mine16 = mine > 0 ? (mine + 15) / 16 * 16 : 16;
    const int blocks = block_of(side16 / 8, 0);
    // what a cluster does not add up of G, beyond the matrix
    if (ctas > 1 && side16 < 128) {
        for (int i = int(threadIdx.x); i < int(2 * kPlane / 16); i += kSmallThreads) {
            reinterpret_cast<uint4*>(gs)[i] = make_uint4(0, 0, 0, 0);
            if (fine) reinterpret_cast<uint4*>(gl)[i] = make_uint4(0, 0, 0, 0);
        }
    }
    // D (+)= A B^T over `depth` k; B read K-major, or MN-major (then its rows are k)
    auto issue = [&](uint32_t a, uint32_t b, bool b_mn, int depth, bool add) {
        const uint32_t kind = mma_kind(0, false, b_mn, 128, 128);
        const uint64_t da = operand(a, false), db = operand(b, b_mn, kPlane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t along = uint64_t(i / 4) * (kPlane >> 4) + uint64_t(i % 4) * 2;   // 16 k of rows of 128 bytes
            if (i * 16 < depth) mma<1>(out, da + along, db + (b_mn ? uint64_t(i) * 128 : along), kind, add || i > 0);
        }
    };
    // what all threads have written is there for the tensor cores
    auto ready = [&] {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tmem_before();
        __syncthreads();
        tmem_after();
    };
    auto done = [&] {
        if (warp == 0 && elected()) commit<1>(bar);
        __syncwarp();
        wait.warp(bar, turn);   // a failure is in the status word; the cluster stays together
        turn ^= 1;
        tmem_after();
    };
    for (int step = 0; step < p.steps; ++step) {
        const float a = p.coefs[step][0], b = p.coefs[step][1], q = p.coefs[step][2] * kUnscale;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t to = h * kPlane + unit_at(r, j);
            *reinterpret_cast<uint4*>(xs + to) = Fp16::pack(x + j * 8);
            *reinterpret_cast<uint4*>(xl + to) = left_of(x + j * 8);
        }
        // G
        ready();
        if (warp == 0 && elected()) {
            issue(xa, xa, false, mine16, false);
            if (fine) {
                issue(xa, xla, false, mine16, true);
                issue(xla, xa, false, mine16, true);
            }
        }
        done();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v[32];
            tmem_load(tmem + i * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= kUnscale;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (ctas > 1) {
                    const int across = h * 8 + i * 4 + j;
                    if (across > r / 8) continue;   // above the diagonal
                    unsigned char* to = parts + block_of(r / 8, across) * 256 + r % 8 * 16;
                    *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(v + j * 8);
                    *reinterpret_cast<float4*>(to + 128) = *reinterpret_cast<const float4*>(v + j * 8 + 4);
                    continue;
                }
                const uint32_t to = h * kPlane + unit_at(r, i * 4 + j);
                *reinterpret_cast<uint4*>(gs + to) = Fp16::pack(v + j * 8);
                if (fine) *reinterpret_cast<uint4*>(gl + to) = left_of(v + j * 8);
            }
        }
        if (ctas > 1) {
            cluster_sync();
            if (ctas == 2) add_up<2, FINE>(parts, fine, blocks, rank);
            else if (ctas == 4) add_up<4, FINE>(parts, fine, blocks, rank);
            else add_up<8, FINE>(parts, fine, blocks, rank);
            cluster_sync();
            lay_out(parts + kSums, gs, side16 / 8);
            if (fine) lay_out(parts + kSumsLow, gl, side16 / 8);
        }
        // Q
        ready();
        if (warp == 0 && elected()) {
            issue(ga, ga, false, side16, false);
            if (fine) {
                issue(ga, gla, false, side16, true);
                issue(gla, ga, false, side16, true);
            }
        }
        done();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v[32];
            tmem_load(tmem + i * 32, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float g[8];
                Fp16::unpack(*reinterpret_cast<const uint4*>(gs + h * kPlane + unit_at(r, i * 4 + j)), g);
                if (fine) {
                    float l[8];
                    Fp16::unpack(*reinterpret_cast<const uint4*>(gl + h * kPlane + unit_at(r, i * 4 + j)), l);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] += l[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = fmaf(b, g[e], q * v[j * 8 + e]);
                const uint32_t to = h * kPlane + unit_at(r, i * 4 + j);
                *reinterpret_cast<uint4*>(qs + to) = Fp16::pack(g);
                *reinterpret_cast<uint4*>(ql + to) = left_of(g);
            }
        }
        // X
        ready();
        if (warp == 0 && elected()) {
            issue(qa, xa, true, side16, false);
            issue(qa, xla, true, side16, true);
            issue(qla, xa, true, side16, true);
        }
        done();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v[32];
            tmem_load(tmem + i * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[i * 32 + e] = fmaf(a, x[i * 32 + e], v[e] * kUnscale);
        }
    }

    // ---- the result, or the update
    if (valid > 0 && !skip) {
        char *dst, *param = nullptr;
        int64_t ld;
        int32_t type = ADAMW_DTYPE_FP32;
        float rate = kUnscale, decay = 0.0f;
        if (MUON) {
            const MuonMatrix t = p.in.table[c.s.first + matrix];
            dst = reinterpret_cast<char*>(t.master);
            param = reinterpret_cast<char*>(t.param);
            ld = cols;
            const float lr = p.in.hp->lr;
            decay = 1.0f - lr * p.in.hp->weight_decay;
            rate = -lr * p.rate[k] * kUnscale;
        } else {
            type = p.dst.dtype;
            dst = p.dst.data + matrix * p.dst.batch_stride * (type == ADAMW_DTYPE_FP32 ? 4 : 2);
            ld = p.dst.row_stride;
        }
        auto place = [&](int e) { return wide ? int64_t(r) * ld + at + h * 64 + e : int64_t(at + h * 64 + e) * ld + r; };
        const bool vector = wide && (MUON ? ld % 8 == 0 && (reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(param)) % 16 == 0
                                          : p.dst.vector != 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v[8];
            if (vector && j * 8 + 8 <= valid) {
                const int64_t to = place(j * 8);
                if (MUON) {
                    *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(dst + to * 4);
                    *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(dst + to * 4 + 16);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = MUON ? fmaf(rate, x[j * 8 + e], decay * v[e]) : x[j * 8 + e] * rate;
                store8_any(dst, to, type, true, 8, v);
                if (MUON) store8_any(param, to, ADAMW_DTYPE_BF16, true, 8, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (j * 8 + e >= valid) break;
                    const int64_t to = place(j * 8 + e);
                    float w = x[j * 8 + e] * rate;
                    if (MUON) w = fmaf(rate, x[j * 8 + e], decay * reinterpret_cast<const float*>(dst)[to]);
                    store_as(dst, to, type, w);
                    if (MUON) store_as(param, to, ADAMW_DTYPE_BF16, w);
                }
            }
        }
    }
    tmem_before();
    if (ctas > 1) cluster_sync();   // nobody reads this CTA's memory any more
    __syncthreads();
    tmem_after();
    if (*static_cast<volatile int32_t*>(&ctl.failed)) {
        if (MUON && threadIdx.x == 0) gave_up_on(p.in.nonfinite);
        let_land();
    }
    if (warp == 0) {
        __syncwarp();
        tmem_free<1>(out, 128);
    }
}

template <bool MUON>
using SmallKernel = void (*)(SmallParams<MUON>);
template <bool MUON>
SmallKernel<MUON> small_of(int32_t dtype, bool fine) {
    constexpr int kOther = MUON ? ADAMW_DTYPE_BF16 : ADAMW_DTYPE_FP16;
    if (dtype == ADAMW_DTYPE_FP32) return fine ? small_kernel<MUON, ADAMW_DTYPE_FP32, true> : small_kernel<MUON, ADAMW_DTYPE_FP32, false>;
    if (dtype == ADAMW_DTYPE_BF16) return fine ? small_kernel<MUON, ADAMW_DTYPE_BF16, true> : small_kernel<MUON, ADAMW_DTYPE_BF16, false>;
    return fine ? small_kernel<MUON, kOther, true> : small_kernel<MUON, kOther, false>;
}

// CTAs of a cluster for a shape; 0: too large.
inline int small_ctas(const Shape& s) {
    const int length = s.rows > s.cols ? s.rows : s.cols;
    if (s.side > kSmallSide || length > 128 * kSmallMost) return 0;
    int n = 1;
    while (n * 128 < length) n *= 2;
    return n;
}

// The shapes of `g`, all small, whose norms (of a plan) begin at `first_sum`.
template <bool MUON>
bool launch_small(const Group& g, const int32_t* first_sum, const adamw_ortho_t& o, const float* coefs, int32_t dtype,
                  int sms, int32_t piece, SmallParams<MUON>* p, cudaStream_t st) {
    p->steps = o.steps;
    p->pretend = g_pretend;
    for (int k = 0; k < o.steps; ++k) memcpy(p->coefs[k], coefs + 3 * (k < o.n_coefficients ? k : o.n_coefficients - 1), 12);
    int most = 1;
    int64_t matrices = 0;
    for (int i = 0; i < g.n; ++i) {
        most = std::max(most, small_ctas(g.shapes[i]));
        matrices += g.shapes[i].count;
    }
    // one launch while its CTAs run at a time, though some have nothing to do;
    // else one for each size of cluster
    const bool together = matrices * most <= sms;
    for (int ctas = together ? most : 1; ctas <= most; ctas *= 2) {
        Group part;
        int32_t sums[kMaxShapes];
        int64_t clusters = 0;
        bool fine = false;
        for (int i = 0; i < g.n; ++i) {
            if (!together && small_ctas(g.shapes[i]) != ctas) continue;
            part.shapes[part.n] = g.shapes[i];
            part.buffers[part.n] = Buffers{};
            sums[part.n] = first_sum[i];
            fine = fine || g.shapes[i].fine;
            p->rate[part.n] = g.rate[i];
            p->first_cluster[part.n++] = int32_t(clusters);
            clusters += g.shapes[i].count;
        }
        if (part.n == 0) continue;
        fill_copies(part, sums, piece, &p->in);
        const SmallKernel<MUON> kernel = small_of<MUON>(dtype, fine);
        if (!launched(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmallBytes)),
                      "cudaFuncSetAttribute") ||
            !launched(launch(kernel, uint32_t(clusters * ctas), kSmallThreads, ctas, kSmallBytes, st, *p), "small launch"))
            return false;
    }
    return true;
}

}  // namespace
