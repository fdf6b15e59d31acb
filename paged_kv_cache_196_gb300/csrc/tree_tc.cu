// Tree attention on the tcgen05 tensor cores: pools of 16-bit types.
//
// A CTA takes a run of pieces (tree_plan.cuh): key tiles of 128 keys (8 blocks) against
// the query rows of a group, 128 of them (MT = 1) or 256 (MT = 2: two row tiles, which
// share every key tile).  Per key tile
//   S = Q K^T      (M = 128 rows, N = 128 keys, fp32 in tensor memory)
//   softmax warps  S -> P, written over S: of every 32 keys' columns the first 16 hold
//                  P_hi = t(P) in the pool's type t, the others P_lo = t(P - P_hi), so the
//                  weights keep 16 significant bits with bf16, 22 with fp16 (less below 2^-12 of
//                  the row's largest, kLift).  (A bf16
//                  weight alone would be off by 2^-8 of itself, as much as a bf16 output.  It
//                  would take 160 us for the four long contexts below when two parts took 195.)
//   O += P_hi V + P_lo V   (P from tensor memory)
// THREE: fp32 output of a bf16 pool, where 16 bits of a weight would be what is lost: a third
// part, in the columns of the second O.  Relative error 1.6e-6 where two parts have 2.3e-6 (the tensor
// cores' own sums, which are cut off and not rounded, are 1.1e-6 of it); 7% more time for the ragged
// batch below, 17% and 37% for the trees that take two row tiles otherwise.
// Roles: softmax warps (a thread = a row = a tensor-memory lane), a warp that copies K and V
// tiles into one ring by TMA (each block-table entry becomes one box), a warp per row tile
// that issues its products, a warp that describes the next piece and copies its queries.
// The ring runs on across pieces.
//
// MT = 1: S is double-buffered, so the next tile's scores are computed while the softmax warps
// work on this one's; Q and O are too, so a piece's end overlaps the next piece's beginning.
// A tile that a call's largest group does not fill is filled with copies of its rows (two
// of up to 64 rows, four of up to 32): the tensor core computes all of S at the same cost, and
// each copy's warps take their own keys of the tile and leave zeros as the others' weights,
// so that all four schedulers share the exponentials; the copies' sums meet at the piece's
// end.  MT = 2: each row tile has one S and one O, and works while the other's products run; a
// warp of its own issues each row tile's products, since one takes hundreds of cycles
// from one wait to the next, and the product of half the weights begins while the other half is
// made.  The row tiles end a key tile in turn: side by side they fall into step, and both wait for
// the tensor core at once, then it for both (four long contexts 156 us in turn, 186 side by side).
//
// What bounds it, measured (times with the kernel that adds up cut pairs, 16-bit output, head_dim
// 128, a GPU that copies 6.69 TB/s and multiplies 1.96 PFLOP/s).  MT = 1, 64 sequences of 512 to
// 4096 tokens, 1 to 17 nodes, 32 heads over 8: 114 us; the 92 us of reading K and V at that rate,
// and what a CTA's start (6 us until the first product), the pieces' ends (3 to 4 us each) and the
// adding up (3 to 6) do not hide.  MT = 2, 16 sequences of 1000 to 8000 and 64 nodes: 99.5 us where K
// and V take 47 and one product each of Q K^T and P V 39; four sequences of 32768 to 131072 with
// 26 nodes, 32 heads over 4: 156 us where they take 92 and 65.  There a key tile of 128 takes
// 4200 clocks, 3264 of them products (two row tiles, 8 + 2 x 8 instructions of 65 to 70 clocks each);
// the rest is the chain S, weights, product of one row tile that the other does not cover.
// Loops over the weights stay rolled: unrolled they pass the instruction cache, and every warp
// waits for code.  K and V leave L2 first, so that partial results stay: 114 us for the ragged batch,
// 121 without.
//
// Tensor memory (512 columns): MT = 1: S at 0 and 128, O at 256 and 384, by tile and by piece
// in turn (THREE: one O, the third parts of both S at 384); MT = 2: S_A, S_B, O_A, O_B.
//
// Only tiles that reach into the tree are masked, by the bits of each row's node and of
// those above it.  Their V rows are looked over before the product: a weight of zero does
// not keep out a NaN, so rows behind the sequence become zeros, and so do the
// infinities and NaN of the tree's own rows, which are added at the end to the rows that
// attend them.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"
#include "tree.h"

namespace pkv {
namespace tree {

// A row's reference is its maximum less kLift (log2 units) until a maximum lies kRenew above that
// one; then sums are scaled.  So weights reach 2^(kLift + kRenew).  bf16 has fp32's exponents and no
// lift.  fp16's steps end at 2^-24: without a lift weights below 2^-3 of the largest would lose bits, and
// those below 2^-25, which may be most of a long context under one large score, all of them.  With it a
// weight is off by 2^-34 of the largest at most.  A higher one has to renew sooner: lifts of 7, 9 and
// 11 (15 in all) take 113.8, 114.0 and 118.2 us for the ragged batch below, 165, 170 and 177 for
// the long contexts in fp16.
template <bool F16>
constexpr float kLift = F16 ? 9.0f : 0.0f;
template <bool F16>
constexpr float kRenew = F16 ? 6.0f : 8.0f;
constexpr uint32_t kColO0 = 256, kColThird = 384;

template <int D, int MT>
struct Layout {
    // A tile is 128 rows, in groups of 8 rows: 64 dimensions of them (a swizzle atom of
    // 1 KiB), then the other 64.  So a block is one box of one copy.
    static constexpr int kHalves = D / 64;
    static constexpr int kGroupBytes = 1024 * kHalves;
    static constexpr int kTileBytes = 16 * kGroupBytes;
    static constexpr int kSlots = D == 64 ? 8 : 5;
    static constexpr int kQBufs = MT == 1 ? 2 : 1;  // of MT tiles
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kBars = kRing + kSlots * kTileBytes;
    static constexpr int kSoftmax = 128 * MT;       // threads
    static constexpr int kCopyWarp = 4 * MT, kQWarp = kCopyWarp + 1, kMmaWarp = kCopyWarp + 2;  // one per row tile
    static constexpr int kThreads = kSoftmax + 64 + 32 * MT;
};

// Where 16-byte part c of a row lies in its tile.
template <int D>
KV_DEVICE int tile_offset(int row, int c) {
    return (row >> 3) * (1024 * (D / 64)) + (c >> 3) * 1024 + (row & 7) * 128 + (((c ^ row) & 7) << 4);
}

template <int D, int MT>
struct Shared {
    uint64_t full[Layout<D, MT>::kSlots], empty[Layout<D, MT>::kSlots];
    uint64_t qfull[2], qempty[2];
    uint64_t sfull[2];             // MT = 1: by tile in turn; MT = 2: of a row tile
    uint64_t pfull[MT][2];         // MT = 1: by tile in turn; MT = 2: of a row tile, half the keys each
    uint64_t odone[MT][2];         // of a row tile, by tile in turn: the product of its weights and V is done
    uint64_t oempty[2];            // MT = 1: by piece in turn; MT = 2: of a row tile
    uint64_t vclean[8];            // MT = 2: by key tile that reaches into the tree, in turn
    uint64_t turn[2];              // MT = 2: a row tile's turn to end a key tile, by key tile of the run
    uint64_t done;
    uint32_t tmem;
    int abort;
    uint32_t gone[8];              // by tile in turn: bit i: block i is not there
    int nonfinite[2];              // by piece in turn: number of a piece whose tree holds some in V
    float2 ml[MT == 1 ? 128 : 1];  // MT = 1: reference and sum of each row copy
    Piece piece[2];                // by Q buffer: the piece whose queries it holds; t1 = 0: no more
    uint2 parents[2][32];          // of the piece's tree, 8 nodes a lane (Ancestors)
    PlaceScratch<Layout<D, MT>::kThreads> scratch;
};

// A pipeline wait.  Under a limit of zero a poll that does not suspend the thread (a suspending one may
// last longer than a short run's waits, and none would run out).
template <bool TW>
KV_DEVICE bool pipe_wait(uint64_t *bar, uint32_t parity, int *err) {
    if constexpr (TW)
        if (g_wait_limit_ns == 0) {
            uint32_t done;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(smem_addr(bar)), "r"(parity)
                : "memory");
            if (!done) atomicOr(err, KV_DEVERR_TIMEOUT);
            return done != 0;
        }
    return mbar_wait<TW>(bar, parity, err);
}

KV_DEVICE float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A block's rows: all of the first three dimensions, two groups of 8 rows from `group` on.
KV_DEVICE void tma_load_4d(void *dst, const CUtensorMap *map, int group, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(0), "r"(group), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// One lane of a warp, the same every time.
KV_DEVICE bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// 32 bytes in one store where they are a sector.
KV_DEVICE void store_sector(void *dst, const uint32_t (&y)[8], bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                     "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

// The largest of kCols columns of this thread's tensor-memory lane (NaN left out), found on the way
// out of tensor memory.
template <int kCols>
KV_DEVICE float tmem_max(uint32_t taddr) {
    uint32_t r[kCols];
    float m;
    if constexpr (kCols == 32) {
        asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
                     : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),"=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15]),"=r"(r[16]),"=r"(r[17]),"=r"(r[18]),"=r"(r[19]),"=r"(r[20]),"=r"(r[21]),"=r"(r[22]),"=r"(r[23]),"=r"(r[24]),"=r"(r[25]),"=r"(r[26]),"=r"(r[27]),"=r"(r[28]),"=r"(r[29]),"=r"(r[30]),"=r"(r[31]), "=f"(m)
                     : "r"(taddr));
    } else {
        asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x64.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, %64, [%65];"
                     : "=r"(r[0]),"=r"(r[1]),"=r"(r[2]),"=r"(r[3]),"=r"(r[4]),"=r"(r[5]),"=r"(r[6]),"=r"(r[7]),"=r"(r[8]),"=r"(r[9]),"=r"(r[10]),"=r"(r[11]),"=r"(r[12]),"=r"(r[13]),"=r"(r[14]),"=r"(r[15]),"=r"(r[16]),"=r"(r[17]),"=r"(r[18]),"=r"(r[19]),"=r"(r[20]),"=r"(r[21]),"=r"(r[22]),"=r"(r[23]),"=r"(r[24]),"=r"(r[25]),"=r"(r[26]),"=r"(r[27]),"=r"(r[28]),"=r"(r[29]),"=r"(r[30]),"=r"(r[31]),"=r"(r[32]),"=r"(r[33]),"=r"(r[34]),"=r"(r[35]),"=r"(r[36]),"=r"(r[37]),"=r"(r[38]),"=r"(r[39]),"=r"(r[40]),"=r"(r[41]),"=r"(r[42]),"=r"(r[43]),"=r"(r[44]),"=r"(r[45]),"=r"(r[46]),"=r"(r[47]),"=r"(r[48]),"=r"(r[49]),"=r"(r[50]),"=r"(r[51]),"=r"(r[52]),"=r"(r[53]),"=r"(r[54]),"=r"(r[55]),"=r"(r[56]),"=r"(r[57]),"=r"(r[58]),"=r"(r[59]),"=r"(r[60]),"=r"(r[61]),"=r"(r[62]),"=r"(r[63]), "=f"(m)
                     : "r"(taddr));
    }
    tc::tmem_wait_ld();
    return m;
}

// Two weights as a pair of the 16-bit type and the pair of what that leaves of them: with half a
// step of 2^-8 (bf16) or 2^-11 (fp16) each, what both leave is at most 2^-16 or 2^-22 of a weight; in
// fp16 at least the half step of its smallest numbers, 2^-25 where a row's largest is 2^kLift or more.
// (Cutting bf16 off instead of rounding it takes as long and leaves twice as much.)
template <bool F16>
KV_DEVICE float2 split(float2 e, uint32_t &hi) {  // the rest, exact
    hi = F16 ? tc::pack_f16x2(e.x, e.y) : tc::pack_bf16x2(e.x, e.y);
    const float2 h = F16 ? f16x2_to_float2(hi) : bf16x2_to_float2(hi);
    return __ffma2_rn(h, make_float2(-1.f, -1.f), e);
}
template <bool F16>
KV_DEVICE uint32_t round2(float2 e) {
    return F16 ? tc::pack_f16x2(e.x, e.y) : tc::pack_bf16x2(e.x, e.y);
}

// D (+)= P B over 64 keys: P at p_tmem in steps of 16 keys, 8 columns each, two steps of every
// kGap columns; B (V, MN-major) advances by `step` 16-byte units per 16 keys.
template <int kGap>
KV_DEVICE void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc_first,
                      uint32_t step) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
        "setp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, %5, %5;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, %6;\n\tmov.b64 b, {y, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
        "add.u32 x, %1, %7;\n\tadd.u32 y, y, %6;\n\tmov.b64 b, {y, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
        "add.u32 x, %1, %8;\n\tadd.u32 y, y, %6;\n\tmov.b64 b, {y, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t}" ::"r"(d_tmem),
        "r"(p_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc_first), "r"(step), "n"(kGap), "n"(kGap + 8)
        : "memory");
}

// D (+)= A B^T over 64 dimensions, both K-major.
KV_DEVICE void mma_ss_k64(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                          uint32_t acc_first) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.u32 p, %6, 0;\n\tsetp.eq.u32 t, %6, %6;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %3, 2;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %3, 4;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %3, 6;\n\tmov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc_first)
        : "memory");
}

// The rows of a piece, the same for every role.
struct Rows {
    int node0, nodes;  // of the group
    int before;        // tokens before the tree
    KV_DEVICE Rows(const TreeParams &p, const Piece &pc) {
        node0 = pc.grp * p.plan.group_nodes;
        nodes = min(p.plan.group_nodes, pc.seq.nodes - node0);
        before = pc.seq.len - pc.seq.nodes;
    }
};

// Bits of a row's node and of those above it, 32 nodes a word.
struct Ancestors {
    uint32_t w[kMaxNodes / 32];

    // All lanes of a warp: lane l's parents, of nodes 8 l .. 8 l + 7, as bytes, 255 for none.
    static KV_DEVICE uint2 pack(const int32_t *parents, int nodes, int *err) {
        const int lane = threadIdx.x & 31;
        uint32_t x[2] = {0xffffffffu, 0xffffffffu};
        bool bad = false;
        int up[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = 8 * lane + k;
            up[k] = i >= nodes ? -1 : parents ? __ldg(parents + i) : i - 1;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = 8 * lane + k;
            if (i < nodes && (up[k] < -1 || up[k] >= i)) {
                bad = true;
                up[k] = -1;
            }
            x[k >> 2] = (x[k >> 2] & ~(255u << (8 * (k & 3)))) | (((uint32_t)up[k] & 255u) << (8 * (k & 3)));
        }
        if (bad) atomicOr(err, KV_DEVERR_TREE);
        return make_uint2(x[0], x[1]);
    }
    // All lanes of a warp: each walks up from its node (a negative one: none), with the lanes' parents.
    KV_DEVICE void walk(uint2 parents, int node) {
#pragma unroll
        for (int k = 0; k < kMaxNodes / 32; ++k) w[k] = 0;
        int i = node;
        while (__any_sync(0xffffffffu, i >= 0)) {
            const int at = i >= 0 ? i : 0;
            const uint32_t a = __shfl_sync(0xffffffffu, parents.x, at >> 3);
            const uint32_t b = __shfl_sync(0xffffffffu, parents.y, at >> 3);
            if (i >= 0) {
#pragma unroll
                for (int k = 0; k < kMaxNodes / 32; ++k) w[k] |= (i >> 5) == k ? 1u << (i & 31) : 0u;
                const uint32_t up = ((i & 4 ? b : a) >> (8 * (i & 3))) & 255u;
                i = up == 255u ? -1 : (int)up;
            }
        }
    }
    KV_DEVICE uint32_t word(int at) const {
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < kMaxNodes / 32; ++k) x = at == k ? w[k] : x;
        return x;
    }
    // As key_bits: bits of 32 keys from `key` on, counted from the tree's first token.
    KV_DEVICE uint32_t keys(int key) const {
        if (key <= -32) return 0xffffffffu;
        if (key < 0) return (0xffffffffu >> (32 + key)) | (w[0] << -key);
        return __funnelshift_r(word(key >> 5), word((key >> 5) + 1), key & 31);
    }
};

template <int D, bool F16, int MT, bool TW, bool THREE = false>
__global__ void __launch_bounds__(Layout<D, MT>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
    using L = Layout<D, MT>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    extern __shared__ __align__(1024) char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    char *sQ = smem, *ring = smem + L::kRing;
    auto &sm = *reinterpret_cast<Shared<D, MT> *>(smem + L::kBars);

    if (warp == L::kMmaWarp) {
        tc::tmem_alloc(&sm.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], MT);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.qfull[s], 2);  // the copies, and what the piece is
            // MT = 2: each row tile's last S, and each softmax warp once it has read what the piece is
            mbar_init(&sm.qempty[s], MT == 1 ? 4 : 2 + 8);
            for (int x = 0; x < MT; ++x) {
                mbar_init(&sm.pfull[x][s], 4);
                mbar_init(&sm.odone[x][s], 1);
            }
            mbar_init(&sm.sfull[s], 1);
            mbar_init(&sm.turn[s], 1);
            mbar_init(&sm.oempty[s], 4);
            sm.nonfinite[s] = -1;
        }
        for (int s = 0; s < 8; ++s) mbar_init(&sm.vclean[s], 4);
        mbar_init(&sm.done, MT);
        sm.abort = 0;
        mbar_init_fence();
    }
    if (tid == L::kQWarp * 32) {
        tc::prefetch_tensormap(&tm_q);
        tc::prefetch_tensormap(&tm_k);
        tc::prefetch_tensormap(&tm_v);
    }
    const Place at = place(p.plan, blockIdx.x, sm.scratch, blockIdx.x == 0 ? p.err : nullptr);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem;
    volatile int *abort_flag = &sm.abort;

    if (warp == L::kCopyWarp) {
        // ================================================== K and V tiles
        // (read once, but for a tree's other groups: partial results stay in L2 instead)
        const uint64_t policy = l2_evict_first_policy();
        int slot = 0, phase = 0, turn = 0;
        unsigned issued = 0;
        bool stop = false;
        Pieces pieces;
        pieces.start(p.plan, at, blockIdx.x);
        Piece pc;
        while (!stop && pieces.next(p.plan, pc)) {
            const int32_t *table = p.tables + (size_t)pc.b * p.plan.max_blocks;
            const int blocks = (pc.seq.len + 15) / 16;
            auto fetch = [&](int t) {  // lanes 0-7: the table's entry; -1: none
                const int i = t * 8 + lane;
                return lane < 8 && t < pc.t1 && i < blocks ? __ldg(table + i) : -1;
            };
            int id = fetch(pc.t0), id_next = fetch(pc.t0 + 1);
            for (int t = pc.t0; t < pc.t1; ++t) {
                const int id_later = fetch(t + 2);
                const bool want = lane < 8 && t * 8 + lane < blocks;
                const bool there = id >= 0 && id < p.num_blocks;
                if (want && !there) atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
                const uint32_t gone = __ballot_sync(0xffffffffu, want && !there) & 255u;
                // groups of 8 rows: -2 and -1 lie outside the tensor and read as zeros
                const int y = want && there ? (id * p.plan.hkv + pc.h) * 2 : -2;
#pragma unroll
                for (int is_v = 0; is_v < 2; ++is_v) {
                    if (lane == 0)
                        stop = *abort_flag || (issued >= L::kSlots && !pipe_wait<TW>(&sm.empty[slot], phase ^ 1, p.err));
                    stop = __shfl_sync(0xffffffffu, stop, 0);
                    if (stop) break;
                    char *dst = ring + slot * L::kTileBytes;
                    if (lane == 0) {
                        if (!is_v) sm.gone[turn & 7] = gone;
                        mbar_arrive_expect_tx(&sm.full[slot], L::kTileBytes);
                    }
                    __syncwarp();
                    if (lane < 8)
                        tma_load_4d(dst + lane * 2 * L::kGroupBytes, is_v ? &tm_v : &tm_k, y, &sm.full[slot], policy);
                    ++issued;
                    if (++slot == L::kSlots) slot = 0, phase ^= 1;
                }
                if (stop) break;
                ++turn;
                id = id_next;
                id_next = id_later;
            }
        }
        if (lane == 0) {
            if (stop) *abort_flag = 1;
            // no copy may be in flight into this CTA's shared memory when it ends
            for (int i = 0; i < L::kSlots && i < issued; ++i) {
                if (--slot < 0) slot = L::kSlots - 1, phase ^= 1;
                mbar_wait_drain(&sm.full[slot], phase, p.err);
            }
        }
    } else if (warp == L::kQWarp) {
        // ================================================== pieces and their query rows
        // What a piece is, its tree and its queries, for the other warps: theirs would be
        // round trips to memory at every piece's beginning.  A box holds 64 dimensions of all
        // heads of tile_nodes nodes; rows past the group's last hold anything (no row
        // reaches another one).
        int copied = 0;  // pieces whose queries were asked for
        Pieces pieces;
        pieces.start(p.plan, at, blockIdx.x);
        Piece pc;
        bool ok = true, more = true;
        for (int n = 0; more; ++n) {
            more = pieces.next(p.plan, pc);
            const int buf = n % L::kQBufs;
            if (lane == 0)
                ok = !*abort_flag &&
                     (n < L::kQBufs || pipe_wait<TW>(&sm.qempty[buf], (n / L::kQBufs - 1) & 1, p.err));
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (!more) pc.t0 = pc.t1 = 0;
            if (lane == 0 && more) {
                const Rows r(p, pc);
                const int per_copy = 128 / p.copies;
                const int boxes = MT == 2 ? (r.nodes > p.plan.tile_nodes ? 2 : 1) : p.copies;
                mbar_arrive_expect_tx(&sm.qfull[buf], boxes * L::kHalves * p.plan.tile_nodes * p.g * 128);
                for (int i = 0; i < boxes; ++i) {
                    char *dst = sQ + buf * L::kTileBytes + (MT == 2 ? i * L::kTileBytes : i * per_copy * 128);
                    const int y = pc.seq.q0 + r.node0 + (MT == 2 ? i * p.plan.tile_nodes : 0);
#pragma unroll
                    for (int h = 0; h < L::kHalves; ++h)
                        tc::tma_load_3d(dst + h * (128 * 128), &tm_q, 64 * h, pc.h * p.g, y, &sm.qfull[buf]);
                }
                ++copied;
            }
            if (more)
                sm.parents[buf][lane] = Ancestors::pack(p.parents ? p.parents + pc.seq.q0 : nullptr, pc.seq.nodes, p.err);
            if (lane == 0) sm.piece[buf] = pc;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.qfull[buf]);
                if (!more) mbar_arrive(&sm.qfull[buf]);  // (in place of the copies')
            }
        }
        if (lane == 0 && p.cuts) p.cuts[blockIdx.x] = cut_of(p.plan, at, blockIdx.x, p.g);
        // No copy may be in flight when the CTA ends.  (A buffer that was given anew had its
        // queries read; the end, once told, is in the one after the last piece's.)
        if (lane == 0)
            for (int i = max(0, copied + (ok ? 1 : 0) - L::kQBufs); i < copied; ++i)
                mbar_wait_drain(&sm.qfull[i % L::kQBufs], (i / L::kQBufs) & 1, p.err);
        if (!ok && lane == 0) *abort_flag = 1;
    } else if (warp >= L::kMmaWarp) {
        // ================================================== products
        // The whole warp runs this and one lane of it issues: the operands of a product lie in
        // registers that all lanes share, and values of a single lane's branch have to be
        // moved there one by one (90 clocks a product beside busy softmax warps, 65 this way).
        {
            const bool one = elect_one();
            auto same = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };  // (tells the compiler)
            auto commit = [&](uint64_t *bar) {
                if (one) tc::mma_commit(bar);
            };
            auto arrive = [&](uint64_t *bar) {
                __syncwarp();
                if (one) mbar_arrive(bar);
            };
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xffffffffu, pipe_wait<TW>(bar, parity, p.err));
            };
            constexpr uint32_t idesc_qk = F16 ? tc::idesc_f16_f32(128, 128, false, false)
                                              : tc::idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t idesc_pv = F16 ? tc::idesc_f16_f32(128, D, false, true)
                                              : tc::idesc_bf16_f32(128, D, false, true);
            const uint32_t d_hi = tc::smem_desc_sw128_hi(L::kGroupBytes);
            const uint32_t q_hi = tc::smem_desc_sw128_hi(1024);  // (Q: 128 rows of 64 dimensions, then the others)
            const uint32_t q_lo = tc::smem_desc_sw128_lo(smem_addr(sQ), 16);
            const uint32_t k_lo = tc::smem_desc_sw128_lo(smem_addr(ring), 16);
            const uint32_t v_lo = tc::smem_desc_sw128_lo(smem_addr(ring), 1024);  // (the other 64 dimensions)
            auto issue_s = [&](uint32_t col, int q_tile, int slot) {
                const uint32_t a = same(q_lo + ((q_tile * L::kTileBytes) >> 4)), b = same(k_lo + ((slot * L::kTileBytes) >> 4));
                const uint32_t d = same(tmem + col);
                if (one) {
#pragma unroll
                    for (int h = 0; h < L::kHalves; ++h) mma_ss_k64(d, a + 1024 * h, q_hi, b + 64 * h, d_hi, idesc_qk, h);
                }
            };
            auto issue_pv = [&](uint32_t col_o, uint32_t col_p, int slot, int half, bool first) {  // 64 keys
                constexpr uint32_t step = 2 * L::kGroupBytes / 16;
                const uint32_t b = same(v_lo + ((slot * L::kTileBytes) >> 4) + 4 * step * half);
                const uint32_t d = same(tmem + col_o), w = same(tmem + col_p + 64 * half);
                const uint32_t third = same(tmem + kColThird + col_p / 2 + 32 * half);
                if (one) {
                    mma_pv<32>(d, w, b, d_hi, idesc_pv, !first, step);
                    mma_pv<32>(d, w + 16, b, d_hi, idesc_pv, 1, step);
                    if constexpr (THREE) mma_pv<16>(d, third, b, d_hi, idesc_pv, 1, step);
                }
            };
            bool ok = true;
            // tile t of the run: K in ring position 2 t, V in 2 t + 1
            auto wait_full = [&](unsigned pos) {
                return wait(&sm.full[pos % L::kSlots], (pos / L::kSlots) & 1);
            };
            if constexpr (MT == 1) {
                // S(t + 1) is issued before PV(t), across pieces too.
                unsigned t = 0;       // next PV
                int n = 0;            // its piece
                int t_left = 0;       // tiles of it that are left
                unsigned s = 0;       // next S
                int sn = -1, s_left = 0;
                bool more = true;
                int len[2] = {0, 0};  // tiles of the pieces whose S has begun and whose PV has not ended
                auto next_s = [&]() {  // issues S(s) if there is one
                    if (s_left == 0) {
                        if (!more) return true;
                        ++sn;
                        if (!wait(&sm.qfull[sn & 1], (sn >> 1) & 1)) return false;
                        s_left = len[sn & 1] = sm.piece[sn & 1].t1 - sm.piece[sn & 1].t0;
                        if (!(more = s_left > 0)) return true;
                    }
                    if (!wait_full(2 * s)) return false;
                    tc::fence_after_sync();
                    issue_s((s & 1) * 128, sn & 1, (int)(2 * s % L::kSlots));
                    commit(&sm.sfull[s & 1]);
                    commit(&sm.empty[2 * s % L::kSlots]);
                    --s_left;
                    ++s;
                    return true;
                };
                ok = next_s();
                t_left = len[0];
                bool first = true;
                while (ok && t < s) {
                    if (!(ok = next_s())) break;
                    // (the weights last: between their arrival and their product nothing is left to do)
                    const int slot = (int)((2 * t + 1) % L::kSlots);
                    const int free_at = THREE ? n - 1 : n - 2;  // the piece that had this O before
                    if ((first && free_at >= 0 && !wait(&sm.oempty[free_at & 1], (free_at >> 1) & 1)) ||
                        !wait_full(2 * t + 1) || !wait(&sm.pfull[0][t & 1], (t >> 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t col_o = kColO0 + (THREE ? 0 : 128 * (n & 1));
                    issue_pv(col_o, (t & 1) * 128, slot, 0, first);
                    issue_pv(col_o, (t & 1) * 128, slot, 1, false);
                    commit(&sm.empty[slot]);
                    commit(&sm.odone[0][t & 1]);
                    ++t;
                    first = --t_left == 0;
                    if (first) {
                        ++n;
                        t_left = len[n & 1];
                    }
                }
            } else {
                // A warp per row tile; the product of the first half of a tile's weights begins
                // while the other half is weighed.  Row tiles issue a key tile's products (and the
                // next scores) in turn: products of both side by side would end together, and then
                // neither's softmax would run beside the other's products (four long contexts: 156
                // us in turn, 186 side by side).
                const int x = warp - L::kMmaWarp;
                unsigned t = 0, u = 0;       // key tiles of the run so far, and of the row tile
                unsigned dirty = 0;          // key tiles of the run so far that reached into a tree
                int worked = 0;              // pieces of the row tile
                for (int n = 0; ok; ++n) {
                    if (!(ok = wait(&sm.qfull[0], n & 1))) break;
                    const Piece pc = sm.piece[0];
                    const int tiles = pc.t1 - pc.t0;
                    if (tiles == 0) break;
                    const Rows r(p, pc);
                    const int clean = max(0, r.before / kTile - pc.t0);  // key tiles before the tree's
                    if (x == 1 && r.nodes <= p.plan.tile_nodes) {
                        arrive(&sm.qempty[0]);
                        for (int i = 0; i < 2 * tiles; ++i) {
                            if (!(ok = wait_full(2 * t + i))) break;
                            arrive(&sm.empty[(2 * t + i) % L::kSlots]);
                            if (i & 1) {
                                if (!(ok = wait(&sm.turn[1], (t + (i >> 1)) & 1))) break;
                                arrive(&sm.turn[0]);
                            }
                        }
                        t += tiles;
                        dirty += max(0, tiles - clean);
                        continue;
                    }
                    auto next_s = [&](int j) {  // tile j of the piece
                        const int slot = (int)(2 * (t + j) % L::kSlots);
                        issue_s(128 * x, x, slot);
                        commit(&sm.sfull[x]);
                        commit(&sm.empty[slot]);
                        if (j + 1 == tiles) commit(&sm.qempty[0]);
                    };
                    if (!(ok = wait_full(2 * t))) break;
                    tc::fence_after_sync();
                    next_s(0);
                    for (int j = 0; j < tiles; ++j, ++u) {
                        // (the weights last: between their arrival and their product nothing is left to do)
                        const int slot = (int)((2 * (t + j) + 1) % L::kSlots);
                        ok = wait_full(2 * (t + j) + 1) && (j + 1 == tiles || wait_full(2 * (t + j) + 2)) &&
                             (j > 0 || worked == 0 || wait(&sm.oempty[x], (worked - 1) & 1));
                        if (ok && j >= clean) {
                            ok = wait(&sm.vclean[dirty & 7], (dirty >> 3) & 1);
                            ++dirty;
                        }
                        for (int half = 0; ok && half < 2; ++half) {
                            if (!(ok = wait(&sm.pfull[x][half], u & 1))) break;
                            if (half == 0 && (x == 1 || t + j > 0) &&
                                !(ok = wait(&sm.turn[x], (t + j + (x == 0)) & 1)))
                                break;
                            tc::fence_after_sync();
                            issue_pv(kColO0 + 128 * x, 128 * x, slot, half, j == 0 && half == 0);
                        }
                        if (!ok) break;
                        if (j + 1 < tiles) next_s(j + 1);
                        arrive(&sm.turn[x ^ 1]);
                        commit(&sm.odone[x][u & 1]);
                        commit(&sm.empty[slot]);
                    }
                    t += tiles;
                    ++worked;
                }
            }
            commit(&sm.done);
            if (!ok) *abort_flag = 1;
            // no product may still write tensor memory when it is freed
            mbar_wait_drain(&sm.done, 0, p.err);
        }
    } else {
        // ================================================== softmax
        const int x = MT == 2 ? warp >> 2 : 0;  // row tile
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int lane_row = tid & 127;
        const int per_copy = 128 / p.copies;
        const int copy = MT == 1 ? lane_row / per_copy : 0;
        const int row = lane_row - copy * per_copy;
        const int row_node = row / p.g, row_head = row - row_node * p.g;
        const int chunks = 4 / p.copies, c0 = copy * chunks, c1 = c0 + chunks;  // of 32 keys, this copy's
        unsigned t = 0;      // key tiles of this row tile so far
        unsigned run_t = 0;  // key tiles of the run so far
        unsigned dirty = 0;  // MT = 2: key tiles of the run so far that reached into a tree
        int n = 0;           // pieces
        bool ok = true;
        while (true) {
            ok = pipe_wait<TW>(&sm.qfull[n % L::kQBufs], (n / L::kQBufs) & 1, p.err);
            ok = !__any_sync(0xffffffffu, !ok);
            Piece pc{};
            uint2 parents = make_uint2(0, 0);
            if (ok) {
                pc = sm.piece[n % L::kQBufs];
                parents = sm.parents[n % L::kQBufs][lane];
                if constexpr (MT == 2) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.qempty[0]);
                }
            }
            const Rows r(p, pc);
            const int tiles = pc.t1 - pc.t0;
            if (MT == 2 && tiles > 0 && x == 1 && r.nodes <= p.plan.tile_nodes) {
                run_t += tiles;
                ++n;
                continue;  // (the tree's rows of V are the first row tile's work)
            }
            const int at_node = x * p.plan.tile_nodes + row_node;  // of the group
            const bool valid = tiles > 0 && row_node < p.plan.tile_nodes && at_node < r.nodes;
            const int node = valid ? r.node0 + at_node : -1;
            const bool idle = __all_sync(0xffffffffu, !valid);  // rows of no query
            Ancestors anc;
            if (!idle && pc.t1 * kTile > r.before) anc.walk(parents, node);
            float m_used = -INFINITY, l_sum = 0.f;
            for (int j = 0; j < tiles; ++j, ++t, ++run_t) {
                const int buf = MT == 1 ? (int)(t & 1) : x;
                bool bad = *abort_flag != 0;
                if (!bad) bad = !pipe_wait<TW>(&sm.sfull[buf], (MT == 1 ? t >> 1 : t) & 1, p.err);
                if (__any_sync(0xffffffffu, bad)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const int key0 = (pc.t0 + j) * kTile;
                const bool tail = key0 + kTile > r.before;
                const uint32_t gone = sm.gone[run_t & 7];
                const uint32_t scol = tmem + lane_base + 128 * buf, third = tmem + lane_base + kColThird + 64 * buf;
                bool rescale = false;
                float alpha = 1.f;
                auto arrive = [&](int which) {  // the weights are there
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.pfull[x][which]);
                };
                if (tail && x == 0) {
                    // the rows of V that lie in the tree or behind it
                    const unsigned pos = 2 * run_t + 1;
                    if (__any_sync(0xffffffffu, !pipe_wait<TW>(&sm.full[pos % L::kSlots], (pos / L::kSlots) & 1, p.err))) {
                        ok = false;
                        break;
                    }
                    char *vt = ring + (int)(pos % L::kSlots) * L::kTileBytes;
                    // (as far as their last block: copies of blocks that are not there are zeros)
                    const int row0 = max(0, r.before - key0), row1 = min(128, (pc.seq.len - key0 + 15) & ~15);
                    constexpr uint32_t top = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll 2
                    for (int i = row0 * (D / 8) + tid; i < row1 * (D / 8); i += 128) {
                        const int at_row = i / (D / 8);
                        uint4 *at4 = reinterpret_cast<uint4 *>(vt + tile_offset<D>(at_row, i % (D / 8)));
                        const uint4 v = *at4;
                        uint32_t y[4] = {v.x, v.y, v.z, v.w};
                        bool here = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((y[k] & top) == top) y[k] &= 0xffff0000u, here = true;
                            if ((y[k] >> 16 & top) == top) y[k] &= 0x0000ffffu, here = true;
                        }
                        if (key0 + at_row >= pc.seq.len)
                            *at4 = make_uint4(0u, 0u, 0u, 0u);
                        else if (here)
                            *at4 = make_uint4(y[0], y[1], y[2], y[3]), sm.nonfinite[n & 1] = n;
                    }
                    tc::fence_proxy_async_smem();  // before the tensor core reads them
                    if constexpr (MT == 2) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.vclean[dirty & 7]);
                        ++dirty;
                    }
                }
                if (!idle) {
                    // Loops over chunks of 32 keys are not unrolled, and scores are read twice:
                    // the code of a tile has to stay in the instruction caches.
                    if (tail || gone) {
#pragma unroll 1
                        for (int c = c0; c < c1; ++c) {
                            if (!gone && key0 + 32 * c + 32 <= r.before) continue;
                            uint32_t bits = tail ? anc.keys(key0 + 32 * c - r.before) : 0xffffffffu;
                            if (gone >> (2 * c) & 1) bits &= 0xffff0000u;
                            if (gone >> (2 * c + 1) & 1) bits &= 0x0000ffffu;
                            uint32_t v[32];
                            tc::tmem_ld32(scol + 32 * c, v);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(bits >> k & 1)) v[k] = __float_as_uint(-INFINITY);
                            tc::tmem_st32(scol + 32 * c, v);
                        }
                        tc::tmem_wait_st();
                    }
                    // Scores are read twice, for the maximum (which tensor memory finds) and for the weights,
                    // 32 at a time: all of them in registers at once would unroll into more code than
                    // the instruction caches next to the schedulers hold.
                    float mrow = chunks == 1 ? tmem_max<32>(scol + 32 * c0) : tmem_max<64>(scol + 32 * c0);
                    if (chunks == 4) mrow = fmaxf(mrow, tmem_max<64>(scol + 64));
                    mrow *= p.scale_log2;  // scale > 0
                    // (a reference rounded up and a difference, which is exact: scores past 2^24 have steps of whole
                    // units, and a weight that another rounding let pass 2^16 would be an fp16 infinity)
                    const float lifted = __fadd_ru(mrow, -kLift<F16>);
                    if (m_used == -INFINITY) {
                        m_used = lifted;
                    } else if (mrow - m_used > kLift<F16> + kRenew<F16>) {
                        alpha = ex2(m_used - lifted);
                        m_used = lifted;
                        l_sum *= alpha;
                        rescale = true;
                    }
                    if (__any_sync(0xffffffffu, rescale)) {
                        // O holds the products up to the tile before once that one's are done
                        if (__any_sync(0xffffffffu, !pipe_wait<TW>(&sm.odone[x][(t - 1) & 1], ((t - 1) >> 1) & 1, p.err))) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t ocol = tmem + lane_base + kColO0 + (THREE ? 0 : 128 * (MT == 1 ? n & 1 : x));
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t v[16];
                            tc::tmem_ld16(ocol + 16 * i, v);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
                            tc::tmem_st16(ocol + 16 * i, v);
                        }
                    }
                    uint32_t va[32], vb[32];
                    tc::tmem_ld32(scol + 32 * c0, va);
                    const float ref = m_used == -INFINITY ? 0.f : m_used;
                    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-ref, -ref);
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    auto weigh = [&](uint32_t (&v)[32], int c) {
                        uint32_t w[32], w3[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 xx = __ffma2_rn(
                                make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc2, nm2);
                            const float2 e = make_float2(ex2(xx.x), ex2(xx.y));
                            acc[k & 1] = __fadd2_rn(acc[k & 1], e);
                            const float2 rest = split<F16>(e, w[k]);
                            if constexpr (THREE)
                                w3[k] = round2<F16>(split<F16>(rest, w[16 + k]));
                            else
                                w[16 + k] = round2<F16>(rest);
                        }
                        tc::tmem_st32(scol + 32 * c, w);
                        if constexpr (THREE) tc::tmem_st16(third + 16 * c, w3);
                    };
                    tc::tmem_wait_ld();
#pragma unroll 1
                    for (int c = c0; c < c1; c += 2) {
                        if (c + 1 < c1) tc::tmem_ld32(scol + 32 * (c + 1), vb);
                        weigh(va, c);
                        if (c + 1 == c1) break;
                        tc::tmem_wait_ld();
                        if (c + 2 < c1) tc::tmem_ld32(scol + 32 * (c + 2), va);
                        weigh(vb, c + 1);
                        tc::tmem_wait_ld();
                        if constexpr (MT == 2) arrive(c >> 1);
                    }
                    l_sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    if (MT == 1 && chunks < 4) {  // the other copies' keys
                        uint32_t zero[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) zero[k] = 0;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c)
                            if (c < c0 || c >= c1) {
                                tc::tmem_st32(scol + 32 * c, zero);
                                if constexpr (THREE) {
                                    uint32_t zero16[16];
#pragma unroll
                                    for (int k = 0; k < 16; ++k) zero16[k] = 0;
                                    tc::tmem_st16(third + 16 * c, zero16);
                                }
                            }
                    }
                }
                if constexpr (MT == 1) {
                    arrive(buf);
                } else if (idle) {
                    arrive(0);
                    arrive(1);
                }
            }
            // ---- the piece's end
            if (ok && tiles > 0) {
                const bool bad = !pipe_wait<TW>(&sm.odone[x][(t - 1) & 1], ((t - 1) >> 1) & 1, p.err);
                ok = !__any_sync(0xffffffffu, bad);
            }
            // MT = 1: all warps stay or leave together; they meet once for every piece and for the end
            if constexpr (MT == 1) {
                sm.ml[lane_row] = make_float2(m_used, l_sum);
                ok = !named_bar_or(1, L::kSoftmax, !ok);
            }
            if (!ok || tiles == 0) break;
            tc::fence_after_sync();
            const uint32_t ocol = tmem + lane_base + kColO0 + (THREE ? 0 : 128 * (MT == 1 ? n & 1 : x));
            const bool nonfinite = *reinterpret_cast<volatile int *>(&sm.nonfinite[n & 1]) == n;
            float factor = 1.f;
            if (MT == 1 && p.copies > 1) {
                // the copies of a row share a reference from here on
                float M = -INFINITY;
                for (int c = 0; c < p.copies; ++c) M = fmaxf(M, sm.ml[row + c * per_copy].x);
                const float ref = M == -INFINITY ? 0.f : M;
                float l = 0.f;
                for (int c = 0; c < p.copies; ++c) {
                    const float2 ml = sm.ml[row + c * per_copy];
                    l += ex2(ml.x - ref) * ml.y;
                }
                factor = ex2(m_used - ref);
                m_used = M;
                l_sum = l;
            }
            const size_t orow = valid ? (size_t)(pc.seq.q0 + node) * p.hq + pc.h * p.g + row_head : 0;
            const int slot_row = 128 * x + row;
            const bool seen = l_sum != 0.f;  // a row with a NaN score stays NaN
            if (pc.slot < 0) factor *= seen ? 1.f / l_sum : 0.f;
            float *part = p.partial + (size_t)max(pc.slot, 0) * (128 * MT) * (D + 2);
            const bool aligned32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
            auto store = [&](int strip, const float (&o)[16]) {  // dimensions 16 strip .. 16 strip + 15 of the row
                if (pc.slot >= 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        reinterpret_cast<float4 *>(part)[(4 * strip + k) * (128 * MT) + slot_row] =
                            make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                } else if (p.out_type == KV_F32) {
                    float *dst = static_cast<float *>(p.out) + orow * D + 16 * strip;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(o[8 * k + i]);
                        store_sector(dst + 8 * k, y, aligned32);
                    }
                } else {
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = F16 ? tc::pack_f16x2(o[2 * i], o[2 * i + 1]) : tc::pack_bf16x2(o[2 * i], o[2 * i + 1]);
                    store_sector(static_cast<uint16_t *>(p.out) + orow * D + 16 * strip, y, aligned32);
                }
            };
            if (MT == 2 || p.copies == 1) {
#pragma unroll 1
                for (int i = 0; i < D / 16; i += 2) {
                    uint32_t v[32];
                    tc::tmem_ld32(ocol + 16 * i, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float o[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(v[16 * h + k]) * factor;
                        if (valid) store(i + h, o);
                    }
                }
            } else {
                // Half of the columns at a time, in strips of 16: copy c sums and stores every
                // strip c, c + copies, ..; the others' go through the Q buffer, free by now:
                // box[strip][4][row of the tile] float4.
                float4 *box = reinterpret_cast<float4 *>(sQ + (n & 1) * L::kTileBytes);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (half) named_bar_sync(2, L::kSoftmax);  // the first half was read
#pragma unroll 1
                    for (int i = 0; i < D / 32; ++i) {
                        if (i % p.copies == copy) continue;
                        uint32_t v[16];
                        tc::tmem_ld16(ocol + half * (D / 2) + 16 * i, v);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            box[(4 * i + k) * 128 + lane_row] =
                                make_float4(__uint_as_float(v[4 * k]) * factor, __uint_as_float(v[4 * k + 1]) * factor,
                                            __uint_as_float(v[4 * k + 2]) * factor, __uint_as_float(v[4 * k + 3]) * factor);
                    }
                    named_bar_sync(2, L::kSoftmax);
#pragma unroll 1
                    for (int i = copy; i < D / 32; i += p.copies) {
                        uint32_t v[16];
                        tc::tmem_ld16(ocol + half * (D / 2) + 16 * i, v);
                        tc::tmem_wait_ld();
                        float o[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(v[k]) * factor;
#pragma unroll 1
                        for (int c = 1; c < p.copies; ++c) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 y = box[(4 * i + k) * 128 + ((lane_row + c * per_copy) & 127)];
                                o[4 * k] += y.x, o[4 * k + 1] += y.y, o[4 * k + 2] += y.z, o[4 * k + 3] += y.w;
                            }
                        }
                        if (valid) store(half * (D / 32) + i, o);
                    }
                }
            }
            if (valid && copy == 0) {
                if (pc.slot >= 0)
                    reinterpret_cast<float2 *>(part + (size_t)128 * MT * D)[slot_row] = make_float2(m_used, l_sum);
                else if (p.lse)
                    p.lse[orow] = seen ? (m_used + log2f(l_sum)) * 0.6931471805599453f : -INFINITY;
            }
            // (uniform over the CTA: every warp reads the same word)
            if (MT == 1 && nonfinite) named_bar_sync(2, L::kSoftmax);  // the other copies' stores
            if (nonfinite && valid && copy == 0) {
                // what was kept out of the products, for the rows that attend it
                const int32_t *table = p.tables + (size_t)pc.b * p.plan.max_blocks;
                for (int k = 0; k < pc.seq.nodes; ++k) {
                    const int key = r.before + k;
                    if (!(anc.word(k >> 5) >> (k & 31) & 1) || key < pc.t0 * kTile || key >= pc.t1 * kTile) continue;
                    const int id = __ldg(table + key / 16);
                    if (id < 0 || id >= p.num_blocks) continue;
                    const uint16_t *from = static_cast<const uint16_t *>(p.v) +
                                           (((size_t)id * p.plan.hkv + pc.h) * 16 + key % 16) * D;
#pragma unroll 1
                    for (int d = 0; d < D; ++d) {
                        const float y = F16 ? f16x2_to_float2(from[d]).x : bf16_to_float(from[d]);
                        if (fabsf(y) < INFINITY) continue;
                        if (pc.slot >= 0) {
                            part[((size_t)(d >> 2) * (128 * MT) + slot_row) * 4 + (d & 3)] += y;
                        } else if (p.out_type == KV_F32) {
                            static_cast<float *>(p.out)[orow * D + d] += y;
                        } else {
                            uint16_t *o = static_cast<uint16_t *>(p.out) + orow * D + d;
                            *o = F16 ? float_to_f16_rn(f16x2_to_float2(*o).x + y) : float_to_bf16_rn(bf16_to_float(*o) + y);
                        }
                    }
                }
            }
            tc::fence_before_sync();
            // the box's ordinary accesses before the copy that fills the Q buffer anew
            if (MT == 1 && p.copies > 1) tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.oempty[MT == 1 ? n & 1 : x]);
                if (MT == 1) mbar_arrive(&sm.qempty[n & 1]);
            }
            ++n;
        }
        if (!ok) *abort_flag = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == L::kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

namespace {

template <int D, int MT>
kv_status launch(const TreeParams &pp, bool f16, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t stream) {
    using L = Layout<D, MT>;
    CUtensorMap tq;
    if (!encode_q_map(&tq, pp.q, pp.total_q, pp.hq, pp.g, pp.plan.tile_nodes, D)) return KV_ERR_CUDA;
    constexpr int smem = L::kBars + (int)sizeof(Shared<D, MT>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    auto pick = [&](auto tw) {
        constexpr bool TW = decltype(tw)::value;
        if constexpr (MT == 1)
            if (!f16 && pp.out_type == KV_F32) return tree_tc_kernel<D, false, 1, TW, true>;
        return f16 ? tree_tc_kernel<D, true, MT, TW> : tree_tc_kernel<D, false, MT, TW>;
    };
    auto fn = test_waits_enabled() ? pick(std::true_type{}) : pick(std::false_type{});
    if (kv_status st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))
        return st;
    fn<<<pp.plan.runs, L::kThreads, smem, stream>>>(tq, tk, tv, pp);
    return cuda_status(cudaGetLastError());
}

}  // namespace

kv_status launch_tc(const TreeParams &pp, int d, int rows, bool f16, const CUtensorMap &tk, const CUtensorMap &tv,
                    cudaStream_t stream) {
    if (d == 128)
        return rows == 128 ? launch<128, 1>(pp, f16, tk, tv, stream) : launch<128, 2>(pp, f16, tk, tv, stream);
    return rows == 128 ? launch<64, 1>(pp, f16, tk, tv, stream) : launch<64, 2>(pp, f16, tk, tv, stream);
}

}  // namespace tree

cudaError_t set_wait_limit_tree(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace pkv
