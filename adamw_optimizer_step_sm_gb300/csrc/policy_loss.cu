// policy_loss.cu -- the token losses: the clipped policy loss with its KL
// term, and the preference loss over pairs of sequences, with the gradients
// of the log-probabilities.
//
// Both touch a few floats per token (policy 12 to 28 bytes, preference 9 to
// 13).  Small batches are bound by the latency of their one launch (policy
// loss of 1000 tokens 5.7 us, preference loss of 4 pairs 4.4 us).  Large ones
// are not yet bound by HBM: 2.1M ragged tokens with a reference, entropies and
// per-token advantages take 27 us (61 MB, 2.3 TB/s; count, loss and the zeroing
// before them), 2.1M even ones with less 20 us: about 760 instructions for 128
// tokens issue in half of the cycles, between chains of dependent loads (a
// warp's sequences, then their counts).  1024 pairs of 2048 tokens take 13 us
// (27 MB, 2.0 TB/s), 19 us where ragged: the longest pair's CTA ends last.
#include "losses_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerLane = 4;    // consecutive tokens of a lane
constexpr int kChunk = 32 * kPerLane;  // and of a warp
constexpr int kMaxGrid = 1216; // 8 CTAs for each of a GB300's 152 SMs
constexpr int kSums = 5;       // pg, KL, entropy, clipped, old KL

uint32_t token_grid(int64_t n) {
    const int64_t g = (n + kWarps * kChunk - 1) / (kWarps * kChunk);
    return uint32_t(g < 1 ? 1 : g > kMaxGrid ? kMaxGrid : g);
}

// Up to here one cluster does a whole call in one launch.  Measured (us, one
// cluster / a grid): policy loss of 1024 tokens 4.2 / 9.4, 8192 6.6 / 10.5,
// 16384 8.7 / 10.5, 32768 13.4 / 10.6; preference loss of 8 pairs and 1024
// tokens 4.6 / 4.4 (and one launch less for the host), 8192 5.0 / 5.6, 32768
// 7.5 / 7.7; of 16 pairs and 16384 tokens, two to a CTA, 7.5 / 5.7.  By ragged
// sequences, policy loss with a weight per sequence: 16384 tokens in 64 11.7 /
// 12.3, in 1024 13.9 / 11.1, in 8192 33 / 20; 8192 tokens in 8192 20 / 21; 1024
// tokens in 1024 13.9 / 17.6, in 8192 19.5 / 24, in 16384 22 / 26: the limit on
// the sequences bounds what the cluster zeroes and counts, a limit on their
// ratio to the tokens would serve the case of many of both better.
constexpr int64_t kClusterTokens = 16384, kClusterSequences = 8192, kClusterPairs = 8;
bool in_one_cluster(const adamw_tokens_t* t) {
    return t->n <= kClusterTokens && t->sequences <= kClusterSequences;
}
uint32_t cluster_ctas(int64_t n) {
    uint32_t c = 1;
    while (c < 8 && n > int64_t(c) * kWarps * kChunk) c *= 2;
    return c;
}

// The workspace: the counts; and unless one cluster does the call, the starts
// of the warps' tokens and the CTAs' sums.
int64_t counts_bytes(int64_t sequences) { return (16 + 4 * sequences + 15) / 16 * 16; }
int64_t starts_bytes(int64_t n) { return ((n + kChunk - 1) / kChunk * 4 + 15) / 16 * 16; }

// Counts tokens by sequence (integers: any order gives the same), CTA `cta`
// of `ctas`.  A warp takes 128 consecutive tokens, four to a lane, and leaves
// what it found of their sequences in starts[] (NULL: nowhere).
__device__ __forceinline__ void count_tokens(const Tokens& t, Counts* out, uint32_t* starts, uint32_t cta,
                                             uint32_t ctas) {
    const uint32_t lane = threadIdx.x % 32;
    uint32_t tokens = 0, filled = 0;
    const uint64_t step = uint64_t(ctas) * kWarps * kChunk;
    for (uint64_t at = (uint64_t(cta) * kWarps + threadIdx.x / 32) * kChunk; at < t.n; at += step) {
        const uint32_t base = uint32_t(at), first = base + lane * kPerLane;
        uint32_t bits = t.counting<kPerLane>(first);
        int32_t seq[kPerLane];
        const uint32_t lo = t.starts_until(base);
        if (starts && lane == 0) starts[base / kChunk] = lo;
        t.sequences_of<kPerLane>(lo, base, first, seq);
        // run by run of the lane's tokens; one atomic where the whole warp is
        // in one sequence
        const int32_t s0 = __shfl_sync(0xffffffffu, seq[0], 0);
        const bool one = Tokens::all_of(seq, s0);
        if (__all_sync(0xffffffffu, one || bits == 0)) {
            const uint32_t k = __reduce_add_sync(0xffffffffu, uint32_t(__popc(bits)));
            if (lane == 0 && k && s0 >= 0) {
                tokens += k;
                filled += atomicAdd(&out->sequence[s0], k) == 0;
            }
            continue;
        }
        while (bits) {
            const int j = __ffs(bits) - 1;
            int32_t s = -1;
            uint32_t k = 0;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                if (i == j) s = seq[i];
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                if ((bits >> i & 1) && seq[i] == s) {
                    ++k;
                    bits &= ~(1u << i);
                }
            if (s >= 0) {
                tokens += k;
                filled += atomicAdd(&out->sequence[s], k) == 0;
            }
        }
    }
    // one atomic per CTA: thousands on one address would wait for one another
    __shared__ uint32_t part[2];
    if (threadIdx.x < 2) part[threadIdx.x] = 0;
    __syncthreads();
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    filled = __reduce_add_sync(0xffffffffu, filled);
    if (lane == 0) {
        atomicAdd(&part[0], tokens);
        atomicAdd(&part[1], filled);
    }
    __syncthreads();
    if (threadIdx.x == 0 && part[0]) {
        atomicAdd(&out->tokens, part[0]);
        atomicAdd(&out->filled, part[1]);
    }
}

__global__ void __launch_bounds__(kThreads) count_kernel(Tokens t, Counts* out, uint32_t* starts) {
    dependency_trigger();
    dependency_wait();
    count_tokens(t, out, starts, blockIdx.x, gridDim.x);
}

// The same by one cluster, which zeroes the counts first.
__device__ __forceinline__ void count_in_cluster(const Tokens& t, Counts* out, uint32_t rank, uint32_t size) {
    uint32_t* words = reinterpret_cast<uint32_t*>(out);
    const uint32_t n = 4 + t.sequences;
    for (uint32_t i = rank * kThreads + threadIdx.x; i < n; i += size * kThreads) words[i] = 0;
    cluster_sync();
    count_tokens(t, out, nullptr, rank, size);
    cluster_sync();
}
__global__ void __launch_bounds__(kThreads) count_cluster_kernel(Tokens t, Counts* out) {
    dependency_trigger();
    dependency_wait();
    count_in_cluster(t, out, cluster_rank(), cluster_size());
}

struct PolicyTokens {
    const float *logp, *old_logp, *ref_logp, *advantages, *entropy;
    float *d_logp, *d_entropy, *stats;
    int64_t* counts;
};

// Four tokens of an array from `first` on, those past n as 0.
__device__ __forceinline__ void load4(const float* p, uint32_t first, uint32_t n, bool vector, float (&x)[kPerLane]) {
    if (vector) {
        const float4 v = *reinterpret_cast<const float4*>(p + first);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) x[j] = first + j < n ? p[first + j] : 0.0f;
    }
}
__device__ __forceinline__ void store4(float* p, uint32_t first, uint32_t n, bool vector, const float (&x)[kPerLane]) {
    if (vector) {
        *reinterpret_cast<float4*>(p + first) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int j = 0; j < kPerLane; ++j)
            if (first + j < n) p[first + j] = x[j];
    }
}

// Loss terms and gradients of CTA `cta` of `ctas`, 128 tokens to a warp: a
// lane's loads are all on their way before it looks for its tokens'
// sequences (from starts[], where the count left them).  Threads below kSums
// return the CTA's sums.  aligned: every array is 16-byte aligned.
template <bool EXACT>
__device__ __forceinline__ Sum2 policy_tokens(const Tokens& t, const Policy& P, const PolicyTokens& a,
                                              const Counts* counts, const uint32_t* starts,
                                              uint32_t tokens, uint32_t filled, bool aligned, uint32_t cta,
                                              uint32_t ctas) {
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Sum2 sum[kSums] = {};
    const uint64_t step = uint64_t(ctas) * kWarps * kChunk;
    for (uint64_t at = (uint64_t(cta) * kWarps + warp) * kChunk; at < t.n; at += step) {
        const uint32_t base = uint32_t(at), first = base + lane * kPerLane;
        const bool vector = aligned && uint64_t(first) + kPerLane <= t.n;
        float logp[kPerLane], old[kPerLane], ref[kPerLane] = {}, ent[kPerLane] = {}, adv[kPerLane] = {};
        load4(a.logp, first, t.n, vector, logp);
        load4(a.old_logp, first, t.n, vector, old);
        if (a.ref_logp) load4(a.ref_logp, first, t.n, vector, ref);
        if (a.entropy) load4(a.entropy, first, t.n, vector, ent);
        if (P.per_token) load4(a.advantages, first, t.n, vector, adv);
        const uint32_t bits = t.counting<kPerLane>(first);
        int32_t seq[kPerLane];
        t.sequences_of<kPerLane>(starts ? starts[base / kChunk] : t.starts_until(base), base, first, seq);
        // the weights and advantages of the lane's sequences, mostly one
        float weight[kPerLane], value[kPerLane];
        const bool one = __all_sync(0xffffffffu, Tokens::all_of(seq, seq[0]));
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            if (j > 0 && one) {
                weight[j] = weight[0];
                value[j] = value[0];
                continue;
            }
            const bool in = seq[j] >= 0 && first + j < t.n;
            const uint32_t q = in ? uint32_t(seq[j]) : 0u;
            const uint32_t count = P.reduce == ADAMW_REDUCE_SEQUENCE && in ? __ldcg(&counts->sequence[q]) : 1u;
            weight[j] = token_weight(P.reduce, P.inv_divisor, tokens, filled, count);
            value[j] = !P.per_token && in ? a.advantages[q] : 0.0f;
        }
        float g[kPerLane], gh[kPerLane], v[kSums] = {};
        // every token alike, whether it counts or not: its results are then
        // taken or left, never multiplied (they may be anything)
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            const bool on = (bits >> j & 1) && seq[j] >= 0;
            const float w = on ? weight[j] : 0.0f;
            const PolicyToken k = policy_token(P, logp[j], old[j], a.ref_logp != nullptr, ref[j],
                                               P.per_token ? adv[j] : value[j]);
            const float term[kSums] = {on ? k.pg : 0.0f, on ? k.kl : 0.0f, on ? ent[j] : 0.0f, k.off,
                                       on ? k.old_kl : 0.0f};
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
                if (EXACT) sum[i].add(w * term[i]); else v[i] = fmaf(w, term[i], v[i]);
            }
            g[j] = on ? w * P.grad_scale * k.grad : 0.0f;
            gh[j] = on ? -w * P.grad_scale * P.entropy_coef : 0.0f;
        }
        if (!EXACT) {
#pragma unroll
            for (int k = 0; k < kSums; ++k) sum[k].add(v[k]);
        }
        if (a.d_logp) store4(a.d_logp, first, t.n, vector, g);
        if (a.d_entropy) store4(a.d_entropy, first, t.n, vector, gh);
    }
    // EXACT: error-free throughout; else the lanes' sums as a tree in fp32 (five
    // roundings, which average out over many warps), the warps' and the CTAs'
    // error-free
    __shared__ float2 part[kSums][kWarps];
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        Sum2 s = sum[k];
        if (EXACT) {
            s = warp_sum(s);
        } else {
            s = {s.value(), 0.0f};
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s.hi += __shfl_xor_sync(0xffffffffu, s.hi, d);
        }
        if (lane == 0) part[k][warp] = make_float2(s.hi, s.lo);
    }
    __syncthreads();
    Sum2 s = {};
    if (threadIdx.x < kSums)
        for (int w = 0; w < kWarps; ++w) s.join(part[threadIdx.x][w].x, part[threadIdx.x][w].y);
    return s;
}

__device__ __forceinline__ void policy_result(const Policy& P, const PolicyTokens& a, const float* mean,
                                              uint32_t tokens, uint32_t filled) {
    float loss = mean[0];
    if (P.kl_coef != 0.0f) loss = fmaf(P.kl_coef, mean[1], loss);
    if (P.entropy_coef != 0.0f) loss = fmaf(-P.entropy_coef, mean[2], loss);
    a.stats[0] = loss;
    for (int k = 0; k < kSums; ++k) a.stats[k + 1] = mean[k];
    a.counts[0] = tokens;
    a.counts[1] = filled;
}

// Over a grid: each CTA leaves its five sums and the last one to finish adds
// them up in the CTAs' order.
__global__ void __launch_bounds__(kThreads)
policy_kernel(Tokens t, Policy P, PolicyTokens a, Counts* counts, const uint32_t* starts, float2* partial,
              bool aligned) {
    dependency_trigger();
    dependency_wait();
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t tokens = counts->tokens, filled = counts->filled;
    const Sum2 mine = policy_tokens<false>(t, P, a, counts, starts, tokens, filled, aligned, blockIdx.x, gridDim.x);
    __shared__ bool last;
    if (threadIdx.x < kSums) {
        partial[blockIdx.x * kSums + threadIdx.x] = make_float2(mine.hi, mine.lo);
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&counts->ticket, 1) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    __shared__ float2 part[kSums][kWarps];
    __shared__ float mean[kSums];
    Sum2 all[kSums] = {};
    for (uint32_t b = threadIdx.x; b < gridDim.x; b += kThreads)
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            const float2 p = __ldcg(&partial[b * kSums + k]);
            all[k].join(p.x, p.y);
        }
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        const Sum2 s = warp_sum(all[k]);
        if (lane == 0) part[k][warp] = make_float2(s.hi, s.lo);
    }
    __syncthreads();
    if (threadIdx.x < kSums) {
        Sum2 s = {};
        for (int w = 0; w < kWarps; ++w) s.join(part[threadIdx.x][w].x, part[threadIdx.x][w].y);
        mean[threadIdx.x] = s.value();
    }
    __syncthreads();
    if (threadIdx.x == 0) policy_result(P, a, mean, tokens, filled);
}

// Few tokens: one cluster counts (COUNT), computes and adds up in one launch.
template <bool COUNT>
__global__ void __launch_bounds__(kThreads)
policy_cluster_kernel(Tokens t, Policy P, PolicyTokens a, Counts* counts, bool aligned) {
    dependency_trigger();
    dependency_wait();
    const uint32_t rank = cluster_rank(), size = cluster_size();
    if (COUNT) count_in_cluster(t, counts, rank, size);
    const uint32_t tokens = __ldcg(&counts->tokens), filled = __ldcg(&counts->filled);
    const Sum2 mine = policy_tokens<true>(t, P, a, counts, nullptr, tokens, filled, aligned, rank, size);
    __shared__ float whole[kSums][2];
    __shared__ float mean[kSums];
    if (threadIdx.x < kSums) {
        whole[threadIdx.x][0] = mine.hi;
        whole[threadIdx.x][1] = mine.lo;
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x < kSums) {
        Sum2 s = mine;
        for (uint32_t k = 1; k < size; ++k)
            s.join(load_remote(&whole[threadIdx.x][0], k), load_remote(&whole[threadIdx.x][1], k));
        mean[threadIdx.x] = s.value();
    }
    cluster_sync();   // no CTA ends while its sums are read
    if (rank == 0 && threadIdx.x == 0) policy_result(P, a, mean, tokens, filled);
}

// ------------------------------------------------------------- preference --

struct Preference {
    float beta, margin, smoothing, grad_scale;
    int32_t kind, average, ref;
};

// log(1 + exp(x)) and sigmoid(x), without overflow.
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    return x >= 0.0f ? 1.0f / (1.0f + e) : e / (1.0f + e);
}

// s / n as a pair of floats: the rounded quotient and what it leaves.
__device__ __forceinline__ Sum2 quotient(const Sum2& s, float n) {
    const float v = s.value(), q = v / n;
    if (!isfinite(v)) return {q, 0.0f};
    // v and s - v, both exact, less q n, whose fused difference from v is exact
    const float rest = __fadd_rn(__fsub_rn(s.hi, v), s.lo);
    return {q, __fadd_rn(fmaf(-q, n, v), rest) / n};
}

constexpr int kMaxWarps = 32;

// Tokens of a thread on their way at a time.  Measured (us, 2 / 4 / 8): 4 pairs
// of 500 tokens 4.4 / 4.6 / 5.2, 4096 of 128 14.9 / 16.0 / 18.9, 1024 of 2048
// 13.3 / 13.5 / 13.5, ragged 19.3 / 19.4 / 17.7.
constexpr int kSideUnroll = 2;

// The sum of logp (less the reference's) over the tokens [b, e) that count, a
// thread's share: every width-th from `me` on, kSideUnroll on their way at a time.
__device__ __forceinline__ void sum_side(const Tokens& t, bool has_ref, const float* logp, const float* ref,
                                         int64_t b, int64_t e, uint32_t me, uint32_t width, Sum2& sum,
                                         uint32_t& tokens) {
    for (int64_t i = b + me; i < e; i += kSideUnroll * int64_t(width)) {
        float x[kSideUnroll], r[kSideUnroll];
        bool on[kSideUnroll];
#pragma unroll
        for (int u = 0; u < kSideUnroll; ++u) {
            const int64_t at = i + u * int64_t(width);
            const bool in = at < e;
            on[u] = in && (!t.mask || t.mask[at] != 0);
            x[u] = in ? logp[at] : 0.0f;
            r[u] = in && has_ref ? ref[at] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kSideUnroll; ++u) {
            if (!on[u]) continue;
            sum.add(x[u]);
            if (has_ref) sum.add(-r[u]);  // the difference unrounded
            ++tokens;
        }
    }
}

// A pair's loss, its h, and the derivative with respect to D.
struct PairLoss {
    float loss, h, dD;
};
__device__ __forceinline__ PairLoss pair_loss(const Preference& P, float D) {
    const float h = P.beta * D - P.margin;
    float loss, dD;
    if (P.kind == ADAMW_PREF_SIGMOID) {
        loss = (1.0f - P.smoothing) * softplus(-h) + P.smoothing * softplus(h);
        dD = P.beta * (P.smoothing * sigmoid(h) - (1.0f - P.smoothing) * sigmoid(-h));
    } else if (P.kind == ADAMW_PREF_HINGE) {
        const float u = 1.0f - h;
        loss = u < 0.0f ? 0.0f : u;  // NaN stays
        dD = h < 1.0f ? -P.beta : h >= 1.0f ? 0.0f : h;
    } else {
        const float u = D - 0.5f / P.beta;
        loss = u * u;
        dD = 2.0f * u;
    }
    return {loss, h, dD};
}

struct PairResult {
    float loss, h, D;
};

// One pair by a group of CTAs (SHARED: a cluster; else one): each sums its
// share of the two sequences' log ratios, the group joins them, and every CTA
// writes its share of the gradient.  losses[pair] receives the loss, or with
// LATER the pair's D, for the kernel of the statistics to go on from.
template <bool SHARED, bool LATER>
__device__ __forceinline__ PairResult preference_pair(const Tokens& t, const Preference& P, const float* logp,
                                                      const float* ref, float* losses, float* rewards,
                                                      float* d_logp, uint32_t pair, uint32_t rank,
                                                      uint32_t size) {
    const uint32_t pairs = t.sequences / 2;
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const uint32_t width = size * blockDim.x, me = rank * blockDim.x + threadIdx.x;
    __shared__ float part[2][3][kMaxWarps];
    __shared__ float whole[2][3];
    int64_t begin[2], end[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint32_t seq = pair + (side ? pairs : 0);
        const int64_t b = t.offsets ? t.offsets[seq] : int64_t(seq) * t.length;
        const int64_t e = t.offsets ? t.offsets[seq + 1] : b + t.length;
        // inside the tokens, whatever the offsets hold
        begin[side] = b < 0 ? 0 : b > int64_t(t.n) ? int64_t(t.n) : b;
        end[side] = e < begin[side] ? begin[side] : e > int64_t(t.n) ? int64_t(t.n) : e;
    }
    Sum2 sum[2] = {};
    uint32_t tokens[2] = {};
#pragma unroll
    for (int side = 0; side < 2; ++side)
        sum_side(t, P.ref == ADAMW_REF_TOKEN, logp, ref, begin[side], end[side], me, width, sum[side],
                 tokens[side]);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const Sum2 s = warp_sum(sum[side]);
        const uint32_t k = __reduce_add_sync(0xffffffffu, tokens[side]);
        if (lane == 0) {
            part[side][0][warp] = s.hi;
            part[side][1][warp] = s.lo;
            part[side][2][warp] = __uint_as_float(k);
        }
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        Sum2 s = {};
        uint32_t k = 0;
        for (uint32_t w = 0; w < warps; ++w) {
            s.join(part[threadIdx.x][0][w], part[threadIdx.x][1][w]);
            k += __float_as_uint(part[threadIdx.x][2][w]);
        }
        whole[threadIdx.x][0] = s.hi;
        whole[threadIdx.x][1] = s.lo;
        whole[threadIdx.x][2] = __uint_as_float(k);
    }
    if (SHARED) cluster_sync(); else __syncthreads();
    Sum2 S[2];
    float share[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        Sum2 s = {};
        uint32_t k = 0;
        if (SHARED) {
            for (uint32_t c = 0; c < size; ++c) {
                s.join(load_remote(&whole[side][0], c), load_remote(&whole[side][1], c));
                k += __float_as_uint(load_remote(&whole[side][2], c));
            }
        } else {
            s = {whole[side][0], whole[side][1]};
            k = __float_as_uint(whole[side][2]);
        }
        if (P.ref == ADAMW_REF_SEQUENCE) s.add(-ref[pair + (side ? pairs : 0)]);
        const float n = float(k > 0 ? k : 1);
        share[side] = P.average ? 1.0f / n : 1.0f;
        S[side] = P.average ? quotient(s, n) : s;
    }
    // the records stay until all have read them
    if (SHARED) cluster_sync(); else __syncthreads();
    // the difference of the pairs of floats, rounded once: two long answers'
    // sums are large and may nearly cancel
    Sum2 difference = S[0];
    difference.join(-S[1].hi, -S[1].lo);
    const float D = difference.value();
    const PairLoss l = pair_loss(P, D);
    if (rank == 0 && threadIdx.x == 0) {
        losses[pair] = LATER ? D : l.loss;
        rewards[pair] = P.beta * S[0].value();
        rewards[pairs + pair] = P.beta * S[1].value();
    }
    const float g = P.grad_scale * l.dD / float(pairs);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const float v = (side ? -g : g) * share[side];
#pragma unroll kSideUnroll
        for (int64_t i = begin[side] + me; i < end[side]; i += width)
            d_logp[i] = !t.mask || t.mask[i] != 0 ? v : 0.0f;
    }
    // tokens outside every sequence
    if (t.offsets && pair == 0) {
        for (int64_t i = me; i < begin[0]; i += width) d_logp[i] = 0.0f;
    }
    if (t.offsets && pair == pairs - 1) {
        for (int64_t i = end[1] + me; i < int64_t(t.n); i += width) d_logp[i] = 0.0f;
    }
    return {l.loss, l.h, D};
}

// A cluster (or CTA) per pair.
template <bool SHARED>
__global__ void __launch_bounds__(1024)
preference_kernel(Tokens t, Preference P, const float* logp, const float* ref, float* losses,
                  float* rewards, float* d_logp) {
    dependency_trigger();
    dependency_wait();
    const uint32_t size = SHARED ? cluster_size() : 1, rank = SHARED ? cluster_rank() : 0;
    preference_pair<SHARED, true>(t, P, logp, ref, losses, rewards, d_logp, blockIdx.x / size, rank, size);
}

// The losses and the statistics over the pairs, from each pair's D in losses[].
__global__ void __launch_bounds__(kThreads)
preference_stats_kernel(uint32_t pairs, Preference P, float* losses, float* stats) {
    dependency_trigger();
    dependency_wait();
    Sum2 loss = {}, h = {};
    uint32_t right = 0;
    // four pairs of a thread on their way at a time: the loads before the stores
    constexpr int kPairs = 4;
    for (uint64_t at = threadIdx.x; at < pairs; at += kPairs * kThreads) {
        float D[kPairs];
#pragma unroll
        for (int u = 0; u < kPairs; ++u) {
            const uint64_t i = at + u * kThreads;
            D[u] = i < pairs ? losses[i] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kPairs; ++u) {
            const uint64_t i = at + u * kThreads;
            if (i >= pairs) break;
            const PairLoss l = pair_loss(P, D[u]);
            losses[i] = l.loss;
            loss.add(l.loss);
            h.add(l.h);
            right += D[u] > 0.0f;
        }
    }
    __shared__ float2 part[2][kWarps];
    __shared__ uint32_t rights[kWarps];
    loss = warp_sum(loss);
    h = warp_sum(h);
    right = __reduce_add_sync(0xffffffffu, right);
    if (threadIdx.x % 32 == 0) {
        part[0][threadIdx.x / 32] = make_float2(loss.hi, loss.lo);
        part[1][threadIdx.x / 32] = make_float2(h.hi, h.lo);
        rights[threadIdx.x / 32] = right;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        Sum2 s = {};
        for (int w = 0; w < kWarps; ++w) s.join(part[threadIdx.x][w].x, part[threadIdx.x][w].y);
        stats[threadIdx.x * 2] = s.value() / float(pairs);
    }
    if (threadIdx.x == 2) {
        uint32_t k = 0;
        for (int w = 0; w < kWarps; ++w) k += rights[w];
        stats[1] = float(k) / float(pairs);
    }
}

// Few pairs: one cluster takes them, a CTA each (in turns), and their
// statistics, in one launch.
__global__ void __launch_bounds__(1024)
preference_cluster_kernel(Tokens t, Preference P, const float* logp, const float* ref, float* losses,
                          float* rewards, float* d_logp, float* stats) {
    dependency_trigger();
    dependency_wait();
    const uint32_t size = cluster_size(), rank = cluster_rank(), pairs = t.sequences / 2;
    Sum2 loss = {}, h = {};
    uint32_t right = 0;
    for (uint32_t pair = rank; pair < pairs; pair += size) {
        const PairResult r = preference_pair<false, false>(t, P, logp, ref, losses, rewards, d_logp, pair, 0, 1);
        loss.add(r.loss);
        h.add(r.h);
        right += r.D > 0.0f;
    }
    __shared__ float mine[5];
    if (threadIdx.x == 0) {
        mine[0] = loss.hi;
        mine[1] = loss.lo;
        mine[2] = h.hi;
        mine[3] = h.lo;
        mine[4] = float(right);
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        for (uint32_t k = 1; k < size; ++k) {
            loss.join(load_remote(&mine[0], k), load_remote(&mine[1], k));
            h.join(load_remote(&mine[2], k), load_remote(&mine[3], k));
            right += uint32_t(load_remote(&mine[4], k));
        }
        stats[0] = loss.value() / float(pairs);
        stats[1] = float(right) / float(pairs);
        stats[2] = h.value() / float(pairs);
    }
    cluster_sync();   // no CTA ends while its record is read
}

}  // namespace

namespace adamw {

int check_tokens(const adamw_tokens_t* t) {
    if (!t || t->n < 0 || t->sequences < 0) return ADAMW_ERR_INVALID_ARG;
    if (t->n > kMaxCount || t->sequences > kMaxCount) return ADAMW_ERR_TOO_LARGE;
    if (t->sequences == 0) return t->n == 0 ? ADAMW_OK : ADAMW_ERR_INVALID_ARG;
    if (!t->offsets && t->n % t->sequences != 0) return ADAMW_ERR_INVALID_ARG;
    if (!aligned(t->offsets, 8)) return ADAMW_ERR_MISALIGNED;
    return ADAMW_OK;
}

int check_policy(const adamw_policy_t* p) {
    if (!p) return ADAMW_ERR_INVALID_ARG;
    const bool ok = p->clip_low >= 0.0f && p->clip_low <= 1.0f && p->clip_high >= 0.0f &&
                    std::isfinite(p->clip_high) &&
                    (p->dual_clip == 0.0f || (p->dual_clip > 1.0f && std::isfinite(p->dual_clip))) &&
                    std::isfinite(p->kl_coef) && std::isfinite(p->entropy_coef) &&
                    std::isfinite(p->grad_scale) && p->kl >= ADAMW_KL_K1 && p->kl <= ADAMW_KL_K3 &&
                    p->reduce >= ADAMW_REDUCE_TOKEN && p->reduce <= ADAMW_REDUCE_FIXED &&
                    (p->reduce != ADAMW_REDUCE_FIXED || (p->divisor > 0.0f && std::isfinite(p->divisor))) &&
                    (p->advantage_per_token == 0 || p->advantage_per_token == 1);
    return ok ? ADAMW_OK : ADAMW_ERR_INVALID_ARG;
}

int launch_counts(const adamw_tokens_t* t, const int64_t* targets, int64_t ignore, void* workspace,
                  cudaStream_t st) {
    Counts* c = static_cast<Counts*>(workspace);
    const Tokens k = tokens_of(t, targets, ignore);
    if (in_one_cluster(t))
        return launched(launch(count_cluster_kernel, cluster_ctas(t->n), kThreads, int(cluster_ctas(t->n)), 0, st,
                               k, c), "count launch")
                   ? ADAMW_OK : ADAMW_ERR_CUDA;
    if (!launched(cudaMemsetAsync(c, 0, size_t(counts_bytes(t->sequences)), st), "counts memset"))
        return ADAMW_ERR_CUDA;
    uint32_t* starts = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + counts_bytes(t->sequences));
    return launched(launch(count_kernel, token_grid(t->n), kThreads, 1, 0, st, k, c, starts), "count launch")
               ? ADAMW_OK : ADAMW_ERR_CUDA;
}

int launch_policy(const adamw_tokens_t* t, const adamw_policy_t* p, const int64_t* targets,
                  int64_t ignore, bool counted, const float* logp, const float* old_logp,
                  const float* ref_logp, const float* advantages, const float* entropy, float* stats,
                  int64_t* counts, float* d_logp, float* d_entropy, void* workspace, cudaStream_t st) {
    const Policy P = policy_of(p);
    const PolicyTokens a = {logp, old_logp, ref_logp, advantages, entropy, d_logp, d_entropy, stats, counts};
    const Tokens k = tokens_of(t, targets, ignore);
    Counts* c = static_cast<Counts*>(workspace);
    bool all_aligned = true;
    const void* arrays[] = {logp, old_logp, ref_logp, p->advantage_per_token ? advantages : nullptr, entropy,
                            d_logp, d_entropy};
    for (const void* x : arrays) all_aligned = all_aligned && aligned(x, 16);
    if (in_one_cluster(t)) {
        auto kernel = counted ? policy_cluster_kernel<false> : policy_cluster_kernel<true>;
        return launched(launch(kernel, cluster_ctas(t->n), kThreads, int(cluster_ctas(t->n)), 0, st, k, P, a, c,
                               all_aligned), "policy launch")
                   ? ADAMW_OK : ADAMW_ERR_CUDA;
    }
    if (!counted) {
        const int rc = launch_counts(t, targets, ignore, workspace, st);
        if (rc != ADAMW_OK) return rc;
    }
    char* rest = static_cast<char*>(workspace) + counts_bytes(t->sequences);
    return launched(launch(policy_kernel, token_grid(t->n), kThreads, 1, 0, st, k, P, a, c,
                           reinterpret_cast<const uint32_t*>(rest),
                           reinterpret_cast<float2*>(rest + starts_bytes(t->n)), all_aligned), "policy launch")
               ? ADAMW_OK : ADAMW_ERR_CUDA;
}

}  // namespace adamw

extern "C" int64_t adamw_policy_workspace(int64_t n, int64_t sequences) {
    if (n < 0 || sequences < 0 || n > kMaxCount || sequences > kMaxCount) return 0;
    const adamw_tokens_t t = {n, sequences, nullptr, nullptr};
    return counts_bytes(sequences) + (in_one_cluster(&t) ? 0 : starts_bytes(n) + int64_t(kMaxGrid) * kSums * int64_t(sizeof(float2)));
}

extern "C" int adamw_policy_loss(const adamw_tokens_t* tokens, const adamw_policy_t* policy,
                                 const float* logp, const float* old_logp, const float* ref_logp,
                                 const float* advantages, const float* entropy, float* stats,
                                 int64_t* counts, float* d_logp, float* d_entropy, void* workspace,
                                 adamw_stream_t stream) {
    int rc = adamw::check_tokens(tokens);
    if (rc != ADAMW_OK) return rc;
    rc = adamw::check_policy(policy);
    if (rc != ADAMW_OK) return rc;
    if (!stats || !counts || !workspace || (policy->kl_coef != 0.0f && !ref_logp) ||
        (policy->entropy_coef != 0.0f && (!entropy || !d_entropy)))
        return ADAMW_ERR_INVALID_ARG;
    if (tokens->n > 0 && (!logp || !old_logp || !advantages || !d_logp)) return ADAMW_ERR_INVALID_ARG;
    const void* floats[] = {logp, old_logp, ref_logp, advantages, entropy, stats, d_logp, d_entropy};
    for (const void* p : floats)
        if (!aligned(p, 4)) return ADAMW_ERR_MISALIGNED;
    if (!aligned(counts, 8) || !aligned(workspace, 16)) return ADAMW_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return adamw::launch_policy(tokens, policy, nullptr, 0, false, logp, old_logp, ref_logp, advantages, entropy,
                                stats, counts, d_logp, d_entropy, workspace, st);
}

extern "C" int adamw_preference_loss(const adamw_tokens_t* tokens, const adamw_preference_t* pref,
                                     const float* logp, const float* ref_logp, float* stats,
                                     float* losses, float* rewards, float* d_logp, adamw_stream_t stream) {
    const int rc = adamw::check_tokens(tokens);
    if (rc != ADAMW_OK) return rc;
    if (!pref || tokens->sequences < 2 || tokens->sequences % 2 != 0) return ADAMW_ERR_INVALID_ARG;
    if (!(pref->beta > 0.0f) || !std::isfinite(pref->beta) || !std::isfinite(0.5f / pref->beta) ||
        !std::isfinite(pref->margin) || !std::isfinite(pref->grad_scale) ||
        !(pref->label_smoothing >= 0.0f && pref->label_smoothing <= 0.5f) ||
        pref->kind < ADAMW_PREF_SIGMOID || pref->kind > ADAMW_PREF_IPO ||
        (pref->kind != ADAMW_PREF_SIGMOID && pref->label_smoothing != 0.0f) ||
        (pref->kind == ADAMW_PREF_IPO && pref->margin != 0.0f) || pref->ref < ADAMW_REF_NONE ||
        pref->ref > ADAMW_REF_SEQUENCE)
        return ADAMW_ERR_INVALID_ARG;
    if (!stats || !losses || !rewards || (pref->ref != ADAMW_REF_NONE && !ref_logp) ||
        (tokens->n > 0 && (!logp || !d_logp)))
        return ADAMW_ERR_INVALID_ARG;
    const void* floats[] = {logp, ref_logp, stats, losses, rewards, d_logp};
    for (const void* p : floats)
        if (!aligned(p, 4)) return ADAMW_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t pairs = tokens->sequences / 2;
    const Preference P = {pref->beta, pref->margin, pref->label_smoothing, pref->grad_scale,
                          pref->kind, pref->length_average, pref->ref};
    const Tokens k = tokens_of(tokens, nullptr, 0);
    const int64_t per_pair = tokens->n / pairs;
    // Larger CTAs where a pair is long, 12 tokens to a thread and more.
    // Measured (us, CTAs of 128 / 256): 4096 pairs of 128 tokens 16.1 / 22.8,
    // of 1024 21.1 / 32.0, 1024 ragged pairs of 2048 on average 23.1 / 19.5;
    // 1024 pairs of 2048, 256 / grown at 8 tokens 13.3 / 17.1; 4 of 65536,
    // grown / 256 12.2 / 14.4.
    int block = 128;
    while (block < 1024 && per_pair >= 12 * block) block *= 2;
    if (pairs <= kClusterPairs && tokens->n <= kClusterTokens) {
        int ctas = 1;
        while (ctas < 8 && ctas < pairs) ctas *= 2;
        return launched(launch(preference_cluster_kernel, uint32_t(ctas), block, ctas, 0, st, k, P, logp, ref_logp,
                               losses, rewards, d_logp, stats), "preference launch")
                   ? ADAMW_OK : ADAMW_ERR_CUDA;
    }
    // CTAs per pair: more where pairs are few and long: up to twice the 152 SMs,
    // each with four tokens to a thread and more.  Clusters for a grid that is
    // busy without them cost: 1024 pairs of 2048 tokens 37 us by two CTAs, 13 by
    // one; with a limit of 1216 in place of 304 200 pairs of 8192 take 81 us for
    // 18.  Measured (us, by at least 1 / 4 / 16 tokens to a thread): 2 pairs of
    // 16384 9.8 / 9.8 / 8.4, 16 of 4096 15.4 / 8.0 / 7.2, 40 of 4096 23 / 11.7 /
    // 7.4, 100 of 8192 17.1 / 17.1 / 12.3, 200 of 8192 17.8 in each: 16 would be the
    // better limit of the three.
    int cluster = 1;
    while (cluster < 8 && pairs * cluster < 304 && per_pair >= cluster * 4 * block) cluster *= 2;
    if (pairs * cluster > kMaxCount) return ADAMW_ERR_TOO_LARGE;
    auto kernel = cluster > 1 ? preference_kernel<true> : preference_kernel<false>;
    if (!launched(launch(kernel, uint32_t(pairs * cluster), block, cluster, 0, st, k, P, logp, ref_logp, losses,
                         rewards, d_logp), "preference launch"))
        return ADAMW_ERR_CUDA;
    return launched(launch(preference_stats_kernel, 1u, kThreads, 1, 0, st, uint32_t(pairs), P, losses, stats),
                    "preference statistics launch")
               ? ADAMW_OK : ADAMW_ERR_CUDA;
}
