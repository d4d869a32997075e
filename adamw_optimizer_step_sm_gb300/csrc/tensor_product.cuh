// tensor_product.cuh -- the main loop of the matrix operators: products of
// 16-bit tiles on the tensor cores with fp32 accumulators, as a persistent
// kernel over a list of tiles that a policy describes.
//
//     D[i][j] = sum_k A(i, k) B(j, k)
//
// Each operand lies in memory either with consecutive k ("K-major": rows of
// k) or with consecutive i or j ("MN-major"), which the tensor cores read
// alike, so that no operand is ever transposed.
//
// A unit (one CTA, or a pair on two neighbouring SMs) computes a tile of
// kRows x kCols in steps of 64 k.  Roles, a warp each: TMA loads into a ring
// of stages; one thread issues tcgen05.mma into one of two accumulators in
// tensor memory; four or eight warps read the other one out and hand it to the
// policy, 32 columns of a row to a thread; and where k ends inside a step at an
// element that the next group owns (the ragged sums over tokens), one warp zeroes
// the rest of the step in shared memory.
//
// Bounds: a 256 x 256 x 64 step of a pair takes the tensor cores of its SMs 512
// cycles, and 64 KB of loads.  The pair shares the loads (128 rows of A and 128 of
// B by each SM); tiles of one CTA load half as much again for the same work and
// are for products with few tiles or groups of few rows.  8192^3 in bf16 takes 551 us
// (1996 TFLOP/s, 104 % of the measured burst rate of 1911; the library's product
// 545 us in the same process); larger products are bound by the power limit.
//
// No wait is endless: after about half a second (a wait for a tile's products: and
// 4 us for each of their steps) it gives up, sets the device's status word, and
// every role leaves.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "adamw_matrix.h"
#include "losses_common.cuh"

namespace {

constexpr int kStepK = 64;                  // elements of k in a stage: 128 bytes, one swizzle row
constexpr int kRowsOfCta = 128;             // accumulator rows of a CTA: the lanes of tensor memory
constexpr int kBlock64 = 64;                // columns of a staged block: 32 rows of 128 bytes
constexpr uint32_t kControlRoom = 1024;
// Cycles after which a wait gives up, and what a wait for all products of a tile has
// besides for each step of 64 k: a step takes 500 to 550 of the tensor cores, about
// 1500 at an SM's share of HBM.
constexpr long long kGiveUp = 1000000000ll, kGiveUpStep = 8192;

// ------------------------------------------------------------------ PTX ---

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

// The address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
// `bar` is a cluster address: this CTA's own or another's.  What these order
// beyond the barrier goes through the asynchronous proxy or tensor memory, which
// have fences of their own: at cluster scope, waits and arrivals would each
// order all of the thread's memory (measured: 790 instead of 1520 TFLOP/s).
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// A box of a three-dimensional tensor into this CTA's shared memory; its bytes
// count at `bar`, which may be the other CTA's of the pair.
template <int PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if (PAIR == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// A box of this CTA's shared memory into a tensor; what is outside is left out, but for
// the rest of 16 bytes that a row ends in (measured: it is written).
__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
                 "r"(z), "r"(src) : "memory");
}
// This thread's stores so far have left shared memory / are done.
__device__ __forceinline__ void stores_read() {
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
// All but the last group of them.
__device__ __forceinline__ void stores_read_but_one() {
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns) {
    if (PAIR == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int PAIR>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    if (PAIR == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
template <int PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    if (PAIR == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"(uint32_t(add)) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"(uint32_t(add)) : "memory");
}
// Arrives at `bar` (in both CTAs of a pair) once this thread's products so far
// have been done.
template <int PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (PAIR == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(bar), "h"(uint16_t(3)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// True in one lane of a converged warp.  The instructions for one thread take
// their operands from uniform registers; under a branch on this the compiler
// knows that there is one.
__device__ __forceinline__ bool elected() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: v[c] is column c of the thread's lane.
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at) : "memory");
}

// The same, zeros where nothing was summed.
__device__ __forceinline__ void load_acc(uint32_t at, bool any, float (&v)[32]) {
    if (any) {
        tmem_load(at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    }
}

// A sector of 32 bytes, at a multiple of 32.
struct Sector {
    uint32_t w[8];
};
__device__ __forceinline__ Sector load_sector(const void* p) {
    Sector s;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]), "=r"(s.w[4]), "=r"(s.w[5]), "=r"(s.w[6]), "=r"(s.w[7])
                 : "l"(__cvta_generic_to_global(p)) : "memory");
    return s;
}
// The same at a multiple of 16.
__device__ __forceinline__ Sector load_halves(const void* p) {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store_halves(void* p, const Sector& s) {
    static_cast<uint4*>(p)[0] = make_uint4(s.w[0], s.w[1], s.w[2], s.w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(s.w[4], s.w[5], s.w[6], s.w[7]);
}
__device__ __forceinline__ void store_sector(void* p, const Sector& s) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "r"(s.w[0]),
                 "r"(s.w[1]), "r"(s.w[2]), "r"(s.w[3]), "r"(s.w[4]), "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7])
                 : "memory");
}
// Sixteen values of 16 bits, or eight fp32, in a sector.
template <int DT>
__device__ __forceinline__ Sector pack_sector(const float* v) {
    Sector s;
    if (DT == ADAMW_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s.w[i] = __float_as_uint(v[i]);
    } else {
        const uint4 a = Elem<DT>::pack(v), b = Elem<DT>::pack(v + 8);
        s.w[0] = a.x, s.w[1] = a.y, s.w[2] = a.z, s.w[3] = a.w;
        s.w[4] = b.x, s.w[5] = b.y, s.w[6] = b.z, s.w[7] = b.w;
    }
    return s;
}
template <int DT>
__device__ __forceinline__ void unpack_sector(const Sector& s, float* v) {
    if (DT == ADAMW_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(s.w[i]);
    } else {
        Elem<DT>::unpack(make_uint4(s.w[0], s.w[1], s.w[2], s.w[3]), v);
        Elem<DT>::unpack(make_uint4(s.w[4], s.w[5], s.w[6], s.w[7]), v + 8);
    }
}
// What rows are a multiple of: nothing that helps, 16 bytes or 32.
constexpr int32_t kAnyRows = 0, kHalfRows = 1, kSectorRows = 2;

// 32 values, of which the first n are there, to a row at a multiple of 32 bytes
// (whole) or of 16.
template <int DT>
__device__ __forceinline__ void store_row(char* at, const float (&v)[32], int n, bool whole) {
    constexpr int k = 32 / Elem<DT>::kSize;   // values of a sector
#pragma unroll
    for (int i = 0; i < 32; i += k) {
        if (i + k <= n) {
            if (whole) store_sector(at + i * Elem<DT>::kSize, pack_sector<DT>(v + i));
            else store_halves(at + i * Elem<DT>::kSize, pack_sector<DT>(v + i));
        } else {
#pragma unroll
            for (int e = i; e < i + k; ++e)
                if (e < n) Elem<DT>::store(at, e, v[e]);
        }
    }
}
template <int DT>
__device__ __forceinline__ void load_row(const char* at, float (&v)[32], int n, bool whole) {
    constexpr int k = 32 / Elem<DT>::kSize;
#pragma unroll
    for (int i = 0; i < 32; i += k) {
        if (i + k <= n) {
            const char* p = at + i * Elem<DT>::kSize;
            unpack_sector<DT>(whole ? load_sector(p) : load_halves(p), v + i);
        } else {
#pragma unroll
            for (int e = i; e < i + k; ++e) v[e] = e < n ? Elem<DT>::load(at, e) : 0.0f;
        }
    }
}
__device__ __forceinline__ void store_row(char* at, int32_t dtype, const float (&v)[32], int n, bool whole) {
    if (dtype == ADAMW_DTYPE_BF16) store_row<ADAMW_DTYPE_BF16>(at, v, n, whole);
    else if (dtype == ADAMW_DTYPE_FP16) store_row<ADAMW_DTYPE_FP16>(at, v, n, whole);
    else store_row<ADAMW_DTYPE_FP32>(at, v, n, whole);
}
__device__ __forceinline__ void load_row(const char* at, int32_t dtype, float (&v)[32], int n, bool whole) {
    if (dtype == ADAMW_DTYPE_BF16) load_row<ADAMW_DTYPE_BF16>(at, v, n, whole);
    else if (dtype == ADAMW_DTYPE_FP16) load_row<ADAMW_DTYPE_FP16>(at, v, n, whole);
    else load_row<ADAMW_DTYPE_FP32>(at, v, n, whole);
}
__device__ __forceinline__ void store_as(char* at, int64_t i, int32_t dtype, float v) {
    if (dtype == ADAMW_DTYPE_BF16) Elem<ADAMW_DTYPE_BF16>::store(at, i, v);
    else if (dtype == ADAMW_DTYPE_FP16) Elem<ADAMW_DTYPE_FP16>::store(at, i, v);
    else Elem<ADAMW_DTYPE_FP32>::store(at, i, v);
}
__device__ __forceinline__ float load_as(const char* at, int64_t i, int32_t dtype) {
    return dtype == ADAMW_DTYPE_BF16   ? Elem<ADAMW_DTYPE_BF16>::load(at, i)
           : dtype == ADAMW_DTYPE_FP16 ? Elem<ADAMW_DTYPE_FP16>::load(at, i) : Elem<ADAMW_DTYPE_FP32>::load(at, i);
}

// ------------------------------------------------- operands in shared memory

// A stage's operand of R rows (of i or j) and 64 k.  K-major: R rows of 128
// bytes, one box.  MN-major: R / 64 boxes of 64 k-rows of 128 bytes.  128-byte
// swizzle in both (16-byte units of a row XORed with the row's number modulo
// 8), which TMA writes and the tensor cores read.  The descriptor: address,
// distance of the 64-wide boxes (MN-major only), distance of groups of eight
// 128-byte rows, version 1, swizzle mode 2 (128 bytes).
__device__ __forceinline__ uint64_t operand(uint32_t addr, bool mn, uint32_t box = 64 * 128) {
    const uint64_t lead = mn ? box >> 4 : 1;
    return uint64_t((addr & 0x3ffff) >> 4) | lead << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// What 16 further k add to the descriptor: 32 bytes of each row, or 16 rows.
__device__ __forceinline__ uint64_t operand_step(bool mn) { return mn ? (16 * 128) >> 4 : 32 >> 4; }

// The instruction descriptor: fp32 accumulators, both operands of the type
// (0: fp16, 1: bf16), their layouts, the tile's shape.
__host__ __device__ constexpr uint32_t mma_kind(int bf16, bool a_mn, bool b_mn, int rows, int cols) {
    return 1u << 4 | uint32_t(bf16) << 7 | uint32_t(bf16) << 10 | uint32_t(a_mn) << 15 | uint32_t(b_mn) << 16 |
           uint32_t(cols / 8) << 17 | uint32_t(rows / 16) << 24;
}

// ------------------------------------------------------------- the kernel --

// What a tile needs of its policy.
struct TileLoads {
    const CUtensorMap *a, *b;
    int32_t a_at, b_at;   // first row (of i, of j) of the unit's tile
    int32_t a_z, b_z;     // third coordinate
    int32_t k_at, k_len;  // range of k; k_len 0: the tile is zeros
    bool a_mn, b_mn;      // layouts
    // Operands of two parts each (P::kParts): `part` > 0 is their k, a multiple of 64,
    // and k_len three of it: A B, then a_low B, then A b_low.
    const CUtensorMap *a_low, *b_low;
    int32_t part;
};

struct Control {
    uint64_t full[16], empty[16], tail[16];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t block[8];   // of the epilogue warps: their staged blocks are there
    uint32_t tmem;
    int32_t failed;
};
static_assert(sizeof(Control) <= kControlRoom, "control block");

// One word a device, set by kernels whose waits ran out.
__device__ int32_t g_tile_status;

struct Waiter {
    static constexpr int32_t kPretend = 2;   // to be reported, though no wait has run out
    int32_t* failed;   // the CTA's: 1, a wait has run out
    // the same answer for all of a warp
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity, int k = 0) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity, k));
    }
    // false: given up (here or elsewhere in the CTA).  k: of the products that are
    // waited for
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, int k) const {
        if (barrier_test(bar, parity)) return true;
        const long long start = clock64();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)
                if (barrier_test(bar, parity)) return true;
            if (*static_cast<volatile int32_t*>(failed) == 1) return false;
            if (clock64() - start > kGiveUp + k / kStepK * kGiveUpStep) {
                *static_cast<volatile int32_t*>(failed) = 1;
                return false;
            }
        }
    }
};
// A CTA's end after a wait that ran out.
__device__ __forceinline__ void let_land() {
    if (threadIdx.x == 0) atomicOr(&g_tile_status, 1);
    // copies and products in flight land within microseconds: a
    // millisecond for them before the memory is given back
    for (int k = 0; k < 1000; ++k) __nanosleep(1000);
}

// What a staged epilogue has: a warp's buffers of 32 rows of 128 bytes, in the
// swizzle of the operands (one or two of them, by P::kStaging).
struct Staged {
    unsigned char *one, *two;
    uint32_t bar, turn;   // where boxes to them arrive, and its parity
    int lane, row, col, end;   // the warp's first row, its columns
    uint32_t acc;         // its lanes of the accumulator
    Waiter wait;
};
// Unit j (16 bytes) of the thread's row in a buffer.
__device__ __forceinline__ uint4* unit_of(unsigned char* buffer, int lane, int j) {
    return reinterpret_cast<uint4*>(buffer + lane * 128 + ((j ^ (lane & 7)) << 4));
}

template <int PAIR_, int COLS_>
struct TileShape {
    static constexpr int kPair = PAIR_, kCols = COLS_, kRows = kRowsOfCta * PAIR_;
    static constexpr int kBRows = kCols / kPair;   // rows of B that each CTA loads
    static constexpr uint32_t kABytes = kRowsOfCta * 128, kBBytes = kBRows * 128;
    static constexpr uint32_t kStageBytes = kABytes + kBBytes;
    static constexpr uint32_t kColumns = 2 * kCols;   // of tensor memory
    static_assert(kColumns <= 512 && (kColumns & (kColumns - 1)) == 0, "tile shape");
};
using PairTile = TileShape<2, 256>;     // 256 x 256 by a pair
using WideTile = TileShape<1, 256>;     // 128 x 256 by one CTA
using SmallTile = TileShape<1, 128>;    // 128 x 128 by one CTA

// Which shape a product takes: the one whose list of tiles is done first by this
// estimate, in cycles: a step of 64 k takes `step`, and what a tile's epilogue
// takes beyond its neighbour's products `rest`.  A 128-column product of 16 k
// takes the tensor cores of an SM as long as one of 256 columns (125 cycles
// against 128, measured without loads), so SmallTile has half the rate and wins
// where its tiles are few or its columns fewer than 128.  Measured: 8192^3 551,
// 673 and 970 us in the three shapes; the Gram matrix of 515 x 1031 in three
// matrices 17, 18 and 13 us.  (256 x 128 by a pair took as long as SmallTile
// for twice its columns, and is not kept.)
struct TileChoice {
    int64_t tiles[3];   // of each shape; 0: not to be taken
};
constexpr int kPairShape = 0, kWideShape = 1, kSmallShape = 2;
inline int choose_shape(const TileChoice& c, int64_t steps, int pairs, int sms) {
    const int64_t step[3] = {512, 540, 500}, rest[3] = {4000, 4000, 2500};
    const int units[3] = {pairs, sms, sms};
    int best = -1;
    int64_t least = 0;
    for (int k = 0; k < 3; ++k) {
        if (c.tiles[k] <= 0) continue;
        const int64_t waves = (c.tiles[k] + units[k] - 1) / units[k];
        const int64_t t = waves * std::max(steps * step[k], rest[k]) + rest[k];
        if (best < 0 || t < least) {
            best = k;
            least = t;
        }
    }
    return best < 0 ? kSmallShape : best;
}

template <class P>
constexpr size_t tile_smem() {
    static_assert(P::kWarps == 4 || P::kWarps == 8, "epilogue warps");
    constexpr size_t n = 1024 + P::kRing + P::kWarps * P::kStaging + kControlRoom + P::kTable;
    static_assert(n <= 232448, "shared memory of a CTA");
    return n;
}
template <class P>
constexpr int tile_threads() { return 128 + 32 * P::kWarps; }

// A policy P over a tile shape S:
//   P::Params       kernel arguments;  P::kTail: k may end inside a step;
//                   P::kParts: operands may be sums of two
//   P::kTable       bytes of shared memory for its tables
//   P::kRing        bytes of the ring of stages
//   P::kWarps       epilogue warps, 4 or 8: each 32 of the CTA's 128 rows, all
//                   columns or half of them
//   prepare(p, table)                    all threads, before the first tile
//   tiles(p, table)                      number of tiles
//   loads(p, table, tile, TileLoads&)    operands
//   bf16(p)                              type of the operands
//   Out: what the epilogue keeps of a tile; out<S>(p, table, tile, rank)
//   wanted(p, out, row, col): whether the 32 x 32 block there has anything to store
//   gave_up(p)                           one thread of a CTA, of which a wait ran out
//   pretend(p)                           whether to say so though none did
//   kStaging        bytes of shared memory of an epilogue warp
//   kStaged: the policy takes a tile's epilogue as a whole, through Staged:
//        begin(p, out, staged, col) asks for what the block at `col` reads, before
//        the products are waited for; finish(p, out, staged, any) does the rest
//        (any: k is not empty).  Else:
//   store(p, out, row, col, float (&v)[32]): results of 32 columns from `col` of row
//        `row` of the CTA's part
//   scalar(out), store_one(p, out, row, col, v): whether results go element by
//        element (rows that are not whole vectors), neighbours by neighbouring lanes
// There a thread has a row, and writes whole 32-byte sectors of it.
template <class P, class S>
__global__ void __launch_bounds__(tile_threads<P>(), 1) tile_kernel(const __grid_constant__ typename P::Params p) {
    constexpr int PAIR = S::kPair, kStages = int(P::kRing / S::kStageBytes);
    static_assert(kStages >= 3 && kStages <= 16, "stages");
    extern __shared__ unsigned char raw[];
    // 1024-byte boundary: the swizzle goes by address bits; the same in both CTAs
    unsigned char* base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    unsigned char* ring = base;
    unsigned char* staging = base + P::kRing;
    Control* ctl = reinterpret_cast<Control*>(base + P::kRing + P::kWarps * P::kStaging);
    unsigned char* table = reinterpret_cast<unsigned char*>(ctl) + kControlRoom;

    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    const uint32_t rank = PAIR == 2 ? cluster_rank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            barrier_init(smem_addr(&ctl->full[s]), PAIR);
            barrier_init(smem_addr(&ctl->empty[s]), 1);
            barrier_init(smem_addr(&ctl->tail[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            barrier_init(smem_addr(&ctl->acc_full[a]), 1);
            barrier_init(smem_addr(&ctl->acc_empty[a]), P::kWarps * PAIR);
        }
        for (int k = 0; k < P::kWarps; ++k) barrier_init(smem_addr(&ctl->block[k]), 1);
        ctl->failed = P::pretend(p) ? Waiter::kPretend : 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc<PAIR>(smem_addr(&ctl->tmem), S::kColumns);
    tmem_before();
    if (PAIR == 2) cluster_sync();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = *static_cast<volatile uint32_t*>(&ctl->tmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    P::prepare(p, table);
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int first = int(blockIdx.x) / PAIR, units = int(gridDim.x) / PAIR;
    const int tiles = P::tiles(p, table);
    const Waiter wait = {&ctl->failed};

    if (warp == 0) {
        // ---- loads
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += units) {
            TileLoads w;
            P::loads(p, table, t, w);
            const bool a_mn = w.a_mn, b_mn = w.b_mn;
            const int a_at = w.a_at + int(rank) * kRowsOfCta, b_at = w.b_at + int(rank) * S::kBRows;
            for (int k = 0; k < w.k_len; k += kStepK, ++it) {
                const uint32_t s = it % kStages;
                if (!(ok = wait.warp(smem_addr(&ctl->empty[s]), (it / kStages & 1) ^ 1))) break;
                if (!elected()) continue;
                const bool tail = P::kTail && k + kStepK > w.k_len;
                const uint32_t own = smem_addr(tail ? &ctl->tail[s] : &ctl->full[s]);
                const uint32_t bar = PAIR == 2 && !tail ? in_cta(own, 0) : own;
                barrier_expect(PAIR == 2 && tail ? in_cta(own, rank) : bar, S::kStageBytes);
                const uint32_t a = smem_addr(ring) + s * S::kStageBytes, b = a + S::kABytes;
                int at = w.k_at + k;
                const CUtensorMap *map_a = w.a, *map_b = w.b;
                if (P::kParts && w.part > 0) {
                    const int part = k / w.part;
                    at -= part * w.part;
                    if (part == 1) map_a = w.a_low;
                    if (part == 2) map_b = w.b_low;
                }
                if (a_mn) {
#pragma unroll
                    for (int i = 0; i < kRowsOfCta / 64; ++i)
                        load_box<PAIR>(a + i * 8192, map_a, a_at + i * 64, at, w.a_z, bar);
                } else {
                    load_box<PAIR>(a, map_a, at, a_at, w.a_z, bar);
                }
                if (b_mn) {
#pragma unroll
                    for (int i = 0; i < S::kBRows / 64; ++i)
                        load_box<PAIR>(b + i * 8192, map_b, b_at + i * 64, at, w.b_z, bar);
                } else {
                    load_box<PAIR>(b, map_b, at, b_at, w.b_z, bar);
                }
            }
        }
        // The products' last arrivals: one that came after this CTA's end would
        // reach the barriers of the next kernel's.
        const uint32_t left = it < uint32_t(kStages) ? it : uint32_t(kStages);
        for (uint32_t k = it - left; k < it && ok; ++k) ok = wait.warp(smem_addr(&ctl->empty[k % kStages]), k / kStages & 1);
    } else if (warp == 1 && rank == 0) {
        // ---- products
        uint32_t it = 0, n = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += units) {
            TileLoads w;
            P::loads(p, table, t, w);
            if (w.k_len == 0) continue;
            const bool a_mn = w.a_mn, b_mn = w.b_mn;
            const uint32_t kind = mma_kind(P::bf16(p), a_mn, b_mn, S::kRows, S::kCols);
            const uint32_t acc = n & 1;
            if (!(ok = wait.warp(smem_addr(&ctl->acc_empty[acc]), (n >> 1 & 1) ^ 1))) break;
            tmem_after();
            for (int k = 0; k < w.k_len; k += kStepK, ++it) {
                const uint32_t s = it % kStages;
                if (!(ok = wait.warp(smem_addr(&ctl->full[s]), it / kStages & 1))) break;
                tmem_after();
                const uint32_t at = smem_addr(ring) + s * S::kStageBytes;
                const uint64_t a = operand(at, a_mn), b = operand(at + S::kABytes, b_mn);
                const uint64_t da = operand_step(a_mn), db = operand_step(b_mn);
                // the last step: only as many 16s of k as it has
                const int parts = w.k_len - k >= kStepK ? kStepK / 16 : (w.k_len - k + 15) / 16;
                if (elected()) {
#pragma unroll
                    for (int i = 0; i < kStepK / 16; ++i)
                        if (i < parts) mma<PAIR>(tmem + acc * S::kCols, a + i * da, b + i * db, kind, k + i > 0);
                    commit<PAIR>(smem_addr(&ctl->empty[s]));
                    if (k + kStepK >= w.k_len) commit<PAIR>(smem_addr(&ctl->acc_full[acc]));
                }
                __syncwarp();
            }
            ++n;
        }
        // the epilogues' last arrivals
        for (uint32_t k = n < 2 ? 0 : n - 2; k < n && ok; ++k) ok = wait.warp(smem_addr(&ctl->acc_empty[k & 1]), k >> 1 & 1);
    } else if (P::kTail && warp == 2) {
        // ---- the last step of a tile whose k ends inside it: rows of k
        // beyond the end (another group's, or anything) become zeros in both
        // operands, as 0 x NaN would reach the sum.  MN-major operands only.
        uint32_t it = 0, turns = 0;   // turns: parity of each stage's next tail
        bool ok = true;
        for (int t = first; t < tiles && ok; t += units) {
            TileLoads w;
            P::loads(p, table, t, w);
            const int steps = (w.k_len + kStepK - 1) / kStepK, rest = w.k_len % kStepK;
            it += uint32_t(steps);
            if (rest == 0) continue;
            const uint32_t s = (it - 1) % kStages;
            if (!(ok = wait.warp(smem_addr(&ctl->tail[s]), turns >> s & 1, w.k_len))) break;
            turns ^= 1u << s;
            const int end = (rest + 15) / 16 * 16;   // what the products read
            unsigned char* at = ring + s * S::kStageBytes;
            const int boxes = int(S::kStageBytes / 8192), units16 = (end - rest) * 8;
            for (int i = lane; i < boxes * units16; i += 32)
                *reinterpret_cast<uint4*>(at + i / units16 * 8192 + rest * 128 + i % units16 * 16) = make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) barrier_arrive(in_cta(smem_addr(&ctl->full[s]), 0));
        }
    } else if (warp >= 4) {
        // ---- results
        float* mine = reinterpret_cast<float*>(staging + (warp - 4) * P::kStaging);
        Staged block = {reinterpret_cast<unsigned char*>(mine), reinterpret_cast<unsigned char*>(mine) + 4096,
                        smem_addr(&ctl->block[warp - 4]), 0, lane, warp % 4 * 32, 0, 0, 0, wait};
        uint32_t n = 0;
        bool ok = true;
        // element (row, col) of the 32 x 32 block, its 16-byte units swizzled
        auto place = [&](int row, int col) { return mine + row * 32 + (((col >> 2) ^ (row & 7)) << 2) + (col & 3); };
        for (int t = first; t < tiles && ok; t += units) {
            TileLoads w;
            P::loads(p, table, t, w);
            const typename P::Out out = P::template out<S>(p, table, t, rank);
            const uint32_t acc = n & 1;
            // a warp reaches the 32 lanes of tensor memory of its number modulo 4
            const int row0 = warp % 4 * 32;
            constexpr int kShare = S::kCols / (P::kWarps / 4);   // columns of the warp
            const int c0 = (warp - 4) / 4 * kShare, c1 = c0 + kShare;
            if constexpr (P::kStaged) {
                block.col = c0;
                block.end = c1;
                block.acc = tmem + (uint32_t(row0) << 16) + acc * S::kCols;
                P::begin(p, out, block, c0);
                if (w.k_len > 0) {
                    if (!(ok = wait.warp(smem_addr(&ctl->acc_full[acc]), n >> 1 & 1, w.k_len))) break;
                    tmem_after();
                }
                if (!(ok = P::finish(p, out, block, w.k_len > 0))) break;
            } else {
                const int row = row0 + lane;
                if (w.k_len > 0) {
                    if (!(ok = wait.warp(smem_addr(&ctl->acc_full[acc]), n >> 1 & 1, w.k_len))) break;
                    tmem_after();
                }
                for (int c = c0; c < c1; c += 32) {
                    if (!P::wanted(p, out, row0, c)) continue;
                    float v[32];
                    load_acc(tmem + (uint32_t(row0) << 16) + acc * S::kCols + uint32_t(c), w.k_len > 0, v);
                    P::store(p, out, row, c, v);
                    if (P::scalar(out)) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(place(lane, i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        __syncwarp();
#pragma unroll 4
                        for (int r = 0; r < 32; ++r) P::store_one(p, out, row0 + r, c + lane, *place(r, lane));
                        __syncwarp();
                    }
                }
            }
            if (w.k_len > 0) {
                tmem_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(in_cta(smem_addr(&ctl->acc_empty[acc]), 0));
                ++n;
            }
        }
        __syncwarp();
        if (P::kStaged && elected()) stores_done();
    }
    __syncwarp();
    __syncthreads();
    if (*static_cast<volatile int32_t*>(&ctl->failed)) {
        if (threadIdx.x == 0) P::gave_up(p);
        let_land();
    }
    tmem_before();
    if (PAIR == 2) cluster_sync();   // the other CTA's arrivals, and its reads of this one's memory
    __syncthreads();
    tmem_after();
    if (warp == 2) tmem_free<PAIR>(tmem, S::kColumns);
}

// -------------------------------------------------------------------- host --

// Whether two batches of matrices share an address (by their outer ends).
inline bool overlap(const adamw_matrices_t& a, const adamw_matrices_t& b) {
    auto end = [](const adamw_matrices_t& m) {
        return reinterpret_cast<uintptr_t>(m.data) +
               uintptr_t((m.batch - 1) * m.batch_stride + (m.rows - 1) * m.row_stride + m.cols) * uintptr_t(dtype_size(m.dtype));
    };
    if (a.batch == 0 || a.rows == 0 || a.cols == 0 || b.batch == 0 || b.rows == 0 || b.cols == 0) return false;
    return reinterpret_cast<uintptr_t>(a.data) < end(b) && reinterpret_cast<uintptr_t>(b.data) < end(a);
}

// Whether every element of a batch has a place of its own: matrices one after the other,
// or their rows by turns.
inline bool apart(const adamw_matrices_t& m) {
    if (m.batch == 0 || m.rows == 0 || m.cols == 0) return true;
    if (m.rows > 1 && m.row_stride < m.cols) return false;
    if (m.batch <= 1) return true;
    using Wide = __int128;   // sizes and strides of any product
    const Wide rows = Wide(m.rows - 1) * m.row_stride + m.cols, matrices = Wide(m.batch - 1) * m.batch_stride + m.cols;
    return m.batch_stride >= rows || (m.batch_stride >= m.cols && (m.rows == 1 || m.row_stride >= matrices));
}

// What the rows of all matrices are a multiple of.
inline int32_t rows_at(const adamw_matrices_t& m) {
    const int size = dtype_size(m.dtype);
    auto whole = [&](int bytes) {
        return aligned(m.data, uintptr_t(bytes)) && (m.rows <= 1 || m.row_stride * size % bytes == 0) &&
               (m.batch <= 1 || m.batch_stride * size % bytes == 0);
    };
    return whole(32) ? kSectorRows : whole(16) ? kHalfRows : kAnyRows;
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

inline EncodeTiled encode_tiled() {
    static EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult how = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// The map of a batch of matrices [batch][rows][cols] of 16-bit elements, rows
// `ld` and matrices `stride` elements apart, for boxes of 64 columns (swizzled; or
// fewer, as they are) and `box_rows` rows.  Base 16-byte aligned; ld and stride multiples of 8.
inline bool tensor_map(CUtensorMap* map, bool bf16, const void* data, int64_t batch, int64_t rows, int64_t cols,
                       int64_t ld, int64_t stride, int box_rows, int box_cols = kStepK) {
    const EncodeTiled f = encode_tiled();
    if (!f) {
        adamw::set_cuda_error("cuTensorMapEncodeTiled", "not found in the driver");
        return false;
    }
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(batch)};
    if (ld <= 0 || stride <= 0) {   // rows or matrices that are one and the same are the caller's to tell apart
        adamw::set_cuda_error("tensor map", "strides must be positive");
        return false;
    }
    const cuuint64_t strides[2] = {cuuint64_t(ld) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = f(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void*>(data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         box_cols == kStepK ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return true;
    adamw::set_cuda_error("cuTensorMapEncodeTiled", "refused the layout");
    return false;
}

// SMs of the current device, and how many pairs of CTAs run at a time.
struct TileUnits {
    int sms = 0, pairs = 0;
};

template <class P>
cudaError_t tile_units(TileUnits* u) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&u->sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(u->sms / 2 * 2));
    cfg.blockDim = dim3(tile_threads<P>());
    cfg.dynamicSmemBytes = tile_smem<P>();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, tile_kernel<P, PairTile>, &cfg)) != cudaSuccess) return e;
    u->pairs = n > 0 ? n : 1;
    return cudaSuccess;
}

}  // namespace
