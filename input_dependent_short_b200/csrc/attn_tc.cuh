// Shared pieces of the tensor-core attention kernels (attn_tc_fwd.cu,
// attn_tc_bwd.cu): operand tiles of 128 rows in shared memory, tensor-memory
// loads and stores, and the bounded waits.
//
// An operand tile holds 128 rows of one head as DP / 64 panels of 64 columns:
// each panel one TMA box, rows of 128 bytes with 128-byte swizzle, 16 KB.  The
// same bytes serve as a K-major operand (rows along M or N, the head's elements
// along K) and as an MN-major one (rows along K, the head's elements along N).
// Columns d .. DP-1 lie outside the tensor and arrive as zeros.
#pragma once

#include "attn.cuh"
#include "lowrank_tc.cuh"
#include "tc.cuh"

namespace dsc {
namespace attn_tc {

constexpr int ROWS = 128;                           // rows of an operand tile
constexpr uint32_t PANEL = ROWS * 128;              // bytes of 64 columns
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;

// The products are issued by a whole, converged warp: the waits and addresses
// before them are then uniform values in uniform registers, and one elected
// lane issues.  (Issued from inside an `if (lane == 0)` each product cost about
// 100 cycles of moves between register files, against the 64 it takes to run:
// the tensor cores idled.)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}\n" : "=r"(p));
    return p != 0;
}

// Descriptor of an operand tile at `addr` (K-major, or MN-major with the next 64 columns a panel further); adding
// bytes / 16 moves its start.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lbo) { return tc::smem_desc_sw128(addr, lbo, 1024); }

// Limit of a wait, in cycles: about a second, and more than the whole item that
// some warps wait for when a document has millions of rows.
__device__ __forceinline__ long long wait_limit(const AttnArgs &a) {
    return 2000000000ll + (a.T / ROWS + 1) * (long long)a.group * 16384;
}

// D[tmem] (+)= A[tmem] * B[smem]: A is 128 lanes x 8 columns of packed bf16 pairs per K step.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[128 x 128] = A * B^T over DP columns, both tiles K-major in shared memory.
template <int DP> __device__ __forceinline__ void mma_tiles(uint32_t d_tmem, uint32_t a, uint32_t b) {
    constexpr uint32_t id = tc::idesc_bf16(ROWS, ROWS, 0, 0);
    const uint64_t ad = tile_desc(a, 16), bd = tile_desc(b, 16);
    if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            const uint32_t off = ((uint32_t)(k >> 2) * PANEL + (uint32_t)(k & 3) * 32u) >> 4;
            tc::mma_bf16(d_tmem, ad + off, bd + off, id, k > 0);
        }
    }
}

// D[128 x DP] (+)= A * B: A [128 x 128] bf16 in tensor memory, B a tile with
// its rows along K; K steps K0 .. K1-1 of 16.  HALVES: A's two halves of 64 K
// columns lie 64 tensor-memory columns apart instead of 32.
template <int DP, int K0 = 0, int K1 = ROWS / 16, bool HALVES = false>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool accumulate) {
    constexpr uint32_t id = tc::idesc_bf16(ROWS, DP, 0, 1);
    const uint64_t bd = tile_desc(b, PANEL);
    if (elect_one()) {
#pragma unroll
        for (int k = K0; k < K1; ++k)
            mma_ts(d_tmem, a_tmem + (HALVES ? 64u * (k >> 2) + 8u * (k & 3) : 8u * k), bd + (uint32_t)k * 128u, id, accumulate || k > 0);
    }
}

// The barrier completes one arrival when the warp's products so far are done (by the elected lane that issued them).
__device__ __forceinline__ void commit(uint32_t bar) {
    if (elect_one()) tc::mma_commit(bar);
}

// 32 lanes x 32 columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
                 "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x of a pair on the FMA pipe, for x <= 127 (anything below -126 gives about
// 2^-126: a weight of 10^-38).  x = n + f with n the nearest integer (the sum
// with 1.5 * 2^23 leaves n in the low mantissa bits), 2^f on [-1/2, 1/2] by the
// degree-4 polynomial of least relative error (2.6e-6, by Remez exchange; the
// rounding to bf16 that follows is 2^-9 = 2e-3), n added to the exponent.  A NaN
// stays one up to there, and what the last sum makes of its bits (0x7fffffff +
// 0xff800000) is fp32's largest number, an infinity once rounded to bf16.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ u64 ex2_fma(u64 x) {
    const u64 magic = mk2(12582912.f, 12582912.f);
    x = mk2(max_nan(lo2(x), -126.f), max_nan(hi2(x), -126.f));
    const u64 t = add2(x, magic);
    const u64 f = add2(x, fma2(t, mk2(-1.f, -1.f), magic));
    u64 p = fma2(mk2(0.009570102207362652f, 0.009570102207362652f), f, mk2(0.05591785907745361f, 0.05591785907745361f));
    p = fma2(p, f, mk2(0.240247443318367f, 0.240247443318367f));
    p = fma2(p, f, mk2(0.6931217908859253f, 0.6931217908859253f));
    p = fma2(p, f, mk2(0.9999992847442627f, 0.9999992847442627f));
    const uint32_t a = __float_as_uint(lo2(p)) + (__float_as_uint(lo2(t)) << 23);
    const uint32_t b = __float_as_uint(hi2(p)) + (__float_as_uint(hi2(t)) << 23);
    return mk2(__uint_as_float(a), __uint_as_float(b));
}

// 32 columns of a warp's 32 rows (x: this lane's row), as bf16, rows `stride`
// apart from `g` = row 0 of the warp, column 0; rows >= n and columns >= ncol
// are not written.  Four lanes trade their four 16-byte pieces first, so that
// a store covers 64 consecutive bytes of 8 rows instead of 16 of 32: the
// epilogue of 128 x 128 values took 3700 cycles without, bound by the lines
// each store touched.
__device__ __forceinline__ void store_rows32(bf16 *g, int64_t stride, const float *x, int n, int ncol, int lane) {
    uint4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = make_uint4(pack_bf2(x[8 * i], x[8 * i + 1]), pack_bf2(x[8 * i + 2], x[8 * i + 3]),
                          pack_bf2(x[8 * i + 4], x[8 * i + 5]), pack_bf2(x[8 * i + 6], x[8 * i + 7]));
#pragma unroll
    for (int b = 1; b < 4; b <<= 1) {
        const bool up = lane & b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & b) continue;
            // lanes without bit b keep piece i and get the partner's piece i for i | b; the others the reverse
            const uint4 send = up ? p[i] : p[i | b];
            uint4 got;
            got.x = __shfl_xor_sync(FULL_MASK, send.x, b);
            got.y = __shfl_xor_sync(FULL_MASK, send.y, b);
            got.z = __shfl_xor_sync(FULL_MASK, send.z, b);
            got.w = __shfl_xor_sync(FULL_MASK, send.w, b);
            if (up) p[i] = got;
            else p[i | b] = got;
        }
    }
    // now p[k] is piece lane % 4 of row 4 (lane / 4) + k
    const int r0 = lane & ~3, c = 8 * (lane & 3);
    if (c < ncol) {
        bf16 *o = g + r0 * stride + c;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r0 + k < n) st16(o + k * stride, p[k]);
    }
}

// One operand tile: rows row0 .. row0+127 of head h into `dst`, completing on `bar`.
template <int DP>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int h, int row0, uint32_t bar) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) tc::tma_load_3d(dst + (uint32_t)c * PANEL, map, 64 * c, h, row0, bar);
}

// Zeroes rows n .. 127 of a tile (one warp); the caller fences.
template <int DP> __device__ __forceinline__ void zero_tail(unsigned char *tile, int n, int lane) {
    for (int i = lane; i < (ROWS - n) * 8; i += 32)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
            *reinterpret_cast<uint4 *>(tile + c * PANEL + n * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// 16 bytes of bf16 hold an infinity or a NaN.
__device__ __forceinline__ bool any_nonfinite(const uint4 &x) {
    auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
    return bad(x.x) || bad(x.y) || bad(x.z) || bad(x.w);
}

// ----------------------------------------------------------- work feed ---
// The kernels are persistent: a block takes (tile, head) items off a counter
// until none is left, so the barriers, tensor memory and instruction cache are
// set up once and an item's loads and first products run under the previous
// one's epilogue.  The loading lane draws the items and passes them on through
// FEED_SLOTS slots of shared memory, each read by `readers` warps.  A wait that
// runs out ends the feed for its warp: a slot that was not seen full, or not
// seen empty, is neither read nor written, so no warp works on an item that
// was never there.
constexpr int FEED_SLOTS = 4;

struct Item {
    int start, len, r0;  // AttnTile
    int h;               // head index, -1: no more items
};

struct Feed {
    uint32_t bars;       // full and empty barriers
    Item *items;
    int *head;           // a list made here: its length, then its tiles
    __device__ uint32_t full(int k) const { return bars + 8u * (uint32_t)(k % FEED_SLOTS); }
    __device__ uint32_t empty(int k) const { return bars + 8u * (uint32_t)(FEED_SLOTS + k % FEED_SLOTS); }
    __device__ AttnTile *tiles() const { return reinterpret_cast<AttnTile *>(head + 4); }
    static constexpr uint32_t BYTES = FEED_SLOTS * (16 + sizeof(Item)) + 16 + INLINE_TILES * (sizeof(AttnTile) + 4);
    __device__ Feed(uint32_t sbase, unsigned char *smem, uint32_t off)
        : bars(sbase + off), items(reinterpret_cast<Item *>(smem + off + FEED_SLOTS * 16)),
          head(reinterpret_cast<int *>(items + FEED_SLOTS)) {}
    __device__ void init(int readers) const {
        for (int k = 0; k < FEED_SLOTS; ++k) {
            tc::mbar_init(full(k), 1);
            tc::mbar_init(empty(k), readers);
        }
    }
    // A short list (a.cu), by the block's threads, as k_attn_tiles makes long
    // ones: thread t looks for the t-th tile, then for its rank by cost.  Ends with a barrier.
    __device__ void make_list(const AttnArgs &a, int rows, bool falling, int tid) const {
        if (!a.cu) return;
        int *cost = reinterpret_cast<int *>(tiles() + INLINE_TILES);
        auto clamp = [](int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); };
        const int T = (int)a.T;
        AttnTile t{0, 0, 0, 0};
        int c = -2, total = 0;  // -2: no tile, -1: rows of no document
        if (tid < INLINE_TILES) {
            int first = clamp(a.cu[0], 0, T), last = first;
            for (int s = 0; s < a.n_docs; ++s) {
                const int b = clamp(a.cu[s], 0, T), e = clamp(a.cu[s + 1], b, T), nt = (e - b + rows - 1) / rows;
                const int j = tid - total;
                last = max(last, e);
                if (j >= 0 && j < nt) {
                    t = AttnTile{b, e - b, j * rows, 0};
                    c = falling ? nt - 1 - j : j;
                }
                total += nt;
            }
            if (total > T / rows + a.n_docs + 2) {  // documents that overlap: none at all
                first = last = T;
                total = 0;
                c = -2;
            }
            const int nf = (first + rows - 1) / rows, nb = (T - last + rows - 1) / rows, i = tid - total;
            if (i >= 0 && i < nf + nb) {
                const int s = i < nf ? i * rows : last + (i - nf) * rows;
                t = AttnTile{s, -min(rows, (i < nf ? first : T) - s), 0, 0};
                c = -1;
            }
            total = min(total + nf + nb, INLINE_TILES);
            cost[tid] = c;
        }
        __syncthreads();
        if (tid < INLINE_TILES && c > -2) {
            int rank = 0;
            for (int j = 0; j < total; ++j) rank += cost[j] > c || (cost[j] == c && j < tid);
            tiles()[rank] = t;
            if (tid == 0) *head = total;
        }
        __syncthreads();
    }
    // The loading lane: this block's item k.  Items of a list in memory are drawn from its counter (the first is the
    // block's index), those of a short list dealt out in turn.
    template <typename Wait>
    __device__ Item draw(int k, const AttnArgs &a, int heads, Wait &&wait, const bool &timed_out) const {
        const int i = k == 0 || a.cu ? (int)(blockIdx.x + k * gridDim.x) : (int)gridDim.x + atomicAdd(a.list.next, 1);
        const int tile = i / heads;
        Item it{0, 0, 0, -1};
        if (tile < (a.cu ? *head : *a.list.count)) {
            const AttnTile t = a.cu ? tiles()[tile] : a.list.tiles[tile];
            it = Item{t.start, t.len, t.r0, i % heads};
        }
        if (k >= FEED_SLOTS) wait(empty(k), (uint32_t)((k / FEED_SLOTS - 1) & 1));
        if (timed_out) return Item{0, 0, 0, -1};
        items[k % FEED_SLOTS] = it;
        tc::mbar_arrive(full(k));
        return it;
    }
    // All lanes of a reading warp, which all end the feed when the wait of one has run out.
    template <typename Wait> __device__ Item get(int k, Wait &&wait, bool &timed_out) const {
        wait(full(k), (uint32_t)((k / FEED_SLOTS) & 1));
        timed_out = __any_sync(FULL_MASK, timed_out);
        if (timed_out) return Item{0, 0, 0, -1};
        const Item it = items[k % FEED_SLOTS];
        __syncwarp();
        return it;
    }
    __device__ void done(int k, int lane) const {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty(k));
    }
};

// Tensor map of a [T, heads, d] view with rows `stride` elements apart: boxes of 128 rows x 64 columns of one head.
inline bool rows_map(CUtensorMap *m, const void *base, int64_t T, int heads, int d, int64_t stride) {
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)heads, (uint64_t)T};
    const uint64_t strides[2] = {(uint64_t)d * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, 1, ROWS};
    return lrtc::make_map(m, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

}  // namespace attn_tc
}  // namespace dsc
