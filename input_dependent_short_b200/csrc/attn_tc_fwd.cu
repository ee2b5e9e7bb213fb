// Causal attention over packed documents on the tensor cores (bf16).
//
// A block owns two query tiles of 128 rows and walks their keys in tiles of
// 128, from the diagonal down.  The two tiles are two query heads of one key
// head where the group is even (they share every key and value tile and have
// equal work), else 256 consecutive rows of one head.  While the tensor cores
// work on one query tile, the softmax of the other runs:
//
//   warps 0-3, 4-7   softmax of tile 0 / 1: a thread owns a row.  S is read
//                    from tensor memory, P = 2^(S c - m c) goes back over it
//                    as bf16, the row's sum stays in a register.
//   warp 8           TMA: the query tiles once, then K and V tiles in turn
//                    through a ring
//   warp 9           issues the products: S = Q K^T (both operands in shared
//                    memory) and O += P V (P from tensor memory), the latter in
//                    two parts, as soon as P's first 96 columns are there.  The
//                    order O(0), S(0), O(1), S(1) keeps the two tiles half a
//                    step apart, so that one's softmax has the exponential unit
//                    while the other's products run (issued by a warp per tile,
//                    the tiles fell into step: 1730 -> 2070 us for 16384 tokens)
//   warp 10          looks the diagonal's V tiles over (below)
//
// The running maximum is lazy: a row's O and sum are rescaled only when its
// maximum has risen by a factor of 2^16 of P since its reference was taken, and
// P starts 2^16 below one, so it never exceeds one: O stays below the number of
// keys times the largest |v|, as in the other kernels.  bf16, the sum and O
// (fp32) are as precise at 2^-16 as at 1; a weight of less than 2^-110 of its
// row's largest counts as zero.  (With 2^8 the rows that see few keys on the
// diagonal rescaled on the next tile nearly always, at 2000 cycles.)  A commit
// of S(j) also covers the earlier O += P V(j-1), so the softmax may rescale O
// without a further wait.
//
// Rows outside the document: V's are zeroed in shared memory (0 * NaN would
// reach the sum); K's only meet masked scores.  On the diagonal a masked P is
// an exact zero, but a V row with a NaN or infinity would still reach the rows
// before it: warp 10 finds such rows, zeroes them for the product, and the
// epilogue adds them to the rows that see them.
#include "attn_tc.cuh"

namespace dsc {
namespace attn_tc {

__device__ int g_dsc_status_attn_fwd = 0;

namespace {

constexpr int THREADS = 384;
// Registers a thread: launched with 168 (64512 of the SM's 65536), then dealt out per warpgroup: the two
// softmax warpgroups keep a 128-column row, the third needs few (2 * 128 * 208 + 128 * 80 = 63488).
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 80;
constexpr float HEADROOM = 16.f;  // log2 of the factor by which P may rise before its row is rescaled
constexpr int SPLIT = 96;  // columns of P after which its first products start

template <int DP> struct Fwd {
    static constexpr uint32_t TILE = PANEL * (DP / 64);   // bytes of an operand tile
    static constexpr int SLOTS = DP == 128 ? 5 : 8;       // K/V ring
    static constexpr uint32_t RING = 2 * TILE;            // after the two query tiles
    static constexpr uint32_t BARS = RING + SLOTS * TILE; // barriers
    static constexpr uint32_t BAD = BARS + 320;           // [FEED_SLOTS][2][4] words
    static constexpr uint32_t FEED = BAD + FEED_SLOTS * 32;
    static constexpr uint32_t TOTAL = FEED + Feed::BYTES + 16 + 1024;  // + the allocation's slot, + alignment
};

struct FwdMaps {
    CUtensorMap q, k, v;
};

// a * 0 + c of packed bf16 pairs
__device__ __forceinline__ uint32_t fma_zero(uint32_t a, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0u), "r"(c));
    return d;
}

// max(a, b, c)
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Adds the value rows that were left out of a diagonal tile's product (a bit of
// `mask` each: row j is key key0 + j) to the warp's rows of O in tensor memory,
// where the row sees them: O += 2^(S c + off) v, in fp32 as the product would,
// so the finite elements of such rows are as precise as any.  q: this lane's
// query row; last: the last row of the mask that it sees (-1: none, q is not
// read).  All lanes of the warp.
__device__ __noinline__ void add_rows(const AttnArgs &a, uint32_t tO, const bf16 *q, int hk, int64_t key0, int last,
                                      float c2, float off, const volatile uint32_t *mask) {
    for (int j = 0; j < ROWS; ++j) {
        if (!((mask[j >> 5] >> (j & 31)) & 1u)) continue;
        const bf16 *k = static_cast<const bf16 *>(a.k) + (key0 + j) * a.ks + (int64_t)hk * a.d;
        const bf16 *v = static_cast<const bf16 *>(a.v) + (key0 + j) * a.vs + (int64_t)hk * a.d;
        const bool sees = j <= last;
        float dot = 0.f;
        if (sees)
            for (int e = 0; e < a.d; ++e) dot = fmaf(__bfloat162float(q[e]), __bfloat162float(k[e]), dot);
        const float w = ex2(fmaf(dot, c2, off));
        __syncwarp();
        for (int c = 0; c < a.d; c += 8) {
            float o[8];
            tc::tmem_ld8(tO + c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (sees) o[e] = fmaf(w, __bfloat162float(v[c + e]), o[e]);
            tmem_st8(tO + c, o);
            tmem_wait_st();
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(THREADS, 1)
    k_attn_fwd_tc(const __grid_constant__ FwdMaps maps, const __grid_constant__ AttnArgs a, int heads, int pair_heads) {
    using S = Fwd<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ring: full, empty, raw (a diagonal V before it has been looked over); per query tile: Q full and empty, S full,
    // P's first part and all of it, O full and empty
    const uint32_t bars = sbase + S::BARS;
    auto full = [&](int s) { return bars + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return bars + 64u + 8u * (uint32_t)s; };
    auto raw = [&](int s) { return bars + 128u + 8u * (uint32_t)s; };
    auto qfull = [&](int i) { return bars + 192u + 8u * (uint32_t)i; };
    auto qempty = [&](int i) { return bars + 208u + 8u * (uint32_t)i; };
    auto sfull = [&](int i) { return bars + 224u + 8u * (uint32_t)i; };
    auto phalf = [&](int i) { return bars + 240u + 8u * (uint32_t)i; };
    auto pfull = [&](int i) { return bars + 256u + 8u * (uint32_t)i; };
    auto ofull = [&](int i) { return bars + 272u + 8u * (uint32_t)i; };
    auto oempty = [&](int i) { return bars + 288u + 8u * (uint32_t)i; };
    const Feed feed(sbase, smem, S::FEED);
    volatile uint32_t *bad = reinterpret_cast<uint32_t *>(smem + S::BAD);  // rows of an item's two diagonal V tiles

    if (tid == 0) {
        for (int s = 0; s < S::SLOTS; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(empty(s), 1);
            tc::mbar_init(raw(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(qfull(i), 1);
            tc::mbar_init(qempty(i), 1);
            tc::mbar_init(sfull(i), 1);
            tc::mbar_init(phalf(i), 4);
            tc::mbar_init(pfull(i), 4);
            tc::mbar_init(ofull(i), 1);
            tc::mbar_init(oempty(i), 4);
        }
        feed.init(10);  // softmax warps, the issuing and the checking warp
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&maps.q);
        tc::tma_prefetch_desc(&maps.k);
        tc::tma_prefetch_desc(&maps.v);
    }
    if (warp == 9) {
        tc::tmem_alloc(sbase + S::FEED + Feed::BYTES, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = 0;  // the whole of the tensor memory: the allocation can only start at column 0
    const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 384};
    pdl_wait();
    pdl_trigger();
    feed.make_list(a, pair_heads ? ROWS : 2 * ROWS, false, tid);

    const long long limit = wait_limit(a);
    bool timed_out = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!timed_out && !tc::mbar_wait(bar, parity, limit)) timed_out = true;
    };
    // Query tile i of an item: head h0 (+ i), rows r0 (+ 128 i) of the document; n[i] key tiles (0: absent), J the most.
    // The V tile of step `it` is the diagonal of query tile 0 (of both, for paired heads), of 1, or of none (-1).
    struct Plan {
        int h0, n[2], J;
        __device__ int diag(int it) const {
            const int j = J - 1 - it;
            return j == n[0] - 1 ? 0 : (j == n[1] - 1 ? 1 : -1);
        }
    };
    auto plan = [&](const Item &t) {
        Plan p;
        p.h0 = pair_heads ? 2 * t.h : t.h;
        p.n[0] = t.r0 / ROWS + 1;
        p.n[1] = pair_heads ? p.n[0] : (t.r0 + ROWS < t.len ? p.n[0] + 1 : 0);
        p.J = max(p.n[0], p.n[1]);
        return p;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (warp == 8) {
            if (lane == 0) {
                int u = 0, uses[2] = {0, 0};  // ring tiles and query tiles loaded so far
                for (int k = 0;; ++k) {
                    const Item t = feed.draw(k, a, heads, wait, timed_out);
                    if (t.h < 0) break;
                    if (t.len < 0) continue;
                    const Plan p = plan(t);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (p.n[i]) {
                            if (uses[i]) wait(qempty(i), (uint32_t)((uses[i] - 1) & 1));
                            if (timed_out) break;
                            ++uses[i];
                            tc::mbar_expect_tx(qfull(i), S::TILE);
                            load_rows<DP>(sbase + i * S::TILE, &maps.q, pair_heads ? p.h0 + i : p.h0,
                                          t.start + t.r0 + (pair_heads ? 0 : i * ROWS), qfull(i));
                        }
                    const int hk = p.h0 / a.group;
                    for (int v = 0; v < 2 * p.J; ++v, ++u) {  // K, V of each step in turn
                        const int s = u % S::SLOTS, it = v >> 1;
                        if (u >= S::SLOTS) wait(empty(s), (uint32_t)((u / S::SLOTS - 1) & 1));
                        if (timed_out) break;
                        const uint32_t bar = (v & 1) && p.diag(it) >= 0 ? raw(s) : full(s);
                        tc::mbar_expect_tx(bar, S::TILE);
                        load_rows<DP>(sbase + S::RING + s * S::TILE, v & 1 ? &maps.v : &maps.k, hk,
                                      t.start + (p.J - 1 - it) * ROWS, bar);
                    }
                }
                for (int s = 0; s < S::SLOTS && s < u; ++s) {  // every load has landed before the block may end
                    const int last = s + ((u - 1 - s) / S::SLOTS) * S::SLOTS;
                    tc::mbar_wait(full(s), (uint32_t)((last / S::SLOTS) & 1), limit);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (uses[i]) tc::mbar_wait(qfull(i), (uint32_t)((uses[i] - 1) & 1), limit);
            }
        } else if (warp == 9) {
            int u0 = 0, uses[2] = {0, 0};
            uint32_t ph[2] = {0, 0};
            auto ring = [&](int u) { return sbase + S::RING + (uint32_t)(u % S::SLOTS) * S::TILE; };
            auto ready = [&](int u) {  // tile u of the ring has landed
                wait(full(u % S::SLOTS), (uint32_t)((u / S::SLOTS) & 1));
                tc::fence_after_sync();
            };
            for (int k = 0;; ++k) {
                const Item t = feed.get(k, wait, timed_out);
                feed.done(k, lane);
                if (t.h < 0) break;
                if (t.len < 0) continue;
                const Plan p = plan(t);
                const int J = p.J;
                auto active = [&](int i, int it) { return J - 1 - it < p.n[i]; };
                auto scores = [&](int i, int it) {
                    mma_tiles<DP>(tS[i], sbase + i * S::TILE, ring(u0 + 2 * it));
                    commit(sfull(i));
                    if (it == J - 1) commit(qempty(i));
                };
                ready(u0);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (p.n[i]) wait(qfull(i), (uint32_t)(uses[i] & 1));
                tc::fence_after_sync();
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (active(i, 0)) scores(i, 0);
                commit(empty(u0 % S::SLOTS));
                for (int it = 0; it < J; ++it) {
                    const bool more = it + 1 < J;
                    ready(u0 + 2 * it + 1);
                    if (more) ready(u0 + 2 * it + 2);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (active(i, it)) {
                            const bool first = J - 1 - it == p.n[i] - 1;
                            if (first && uses[i]) wait(oempty(i), (uint32_t)((uses[i] - 1) & 1));
                            wait(phalf(i), ph[i]);
                            tc::fence_after_sync();
                            mma_rows<DP, 0, SPLIT / 16>(tO[i], tS[i], ring(u0 + 2 * it + 1), !first);
                            wait(pfull(i), ph[i]);
                            tc::fence_after_sync();
                            mma_rows<DP, SPLIT / 16>(tO[i], tS[i], ring(u0 + 2 * it + 1), true);
                            ph[i] ^= 1u;
                            if (!more) commit(ofull(i));
                        }
                        if (more && active(i, it + 1)) scores(i, it + 1);
                    }
                    commit(empty((u0 + 2 * it + 1) % S::SLOTS));
                    if (more) commit(empty((u0 + 2 * it + 2) % S::SLOTS));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) uses[i] += p.n[i] > 0;
                u0 += 2 * J;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)  // every product is done
                if (uses[i]) tc::mbar_wait(ofull(i), (uint32_t)((uses[i] - 1) & 1), limit);
        } else if (warp == 10) {
            int u0 = 0;
            uint32_t rp = 0;  // a bit per slot: parity of its raw barrier
            for (int k = 0;; ++k) {
                const Item t = feed.get(k, wait, timed_out);
                if (t.h < 0) break;
                if (t.len < 0) {
                    feed.done(k, lane);
                    continue;
                }
                const Plan p = plan(t);
                volatile uint32_t *rows_bad = bad + (k % FEED_SLOTS) * 8;
                if (lane < 8) rows_bad[lane] = 0;
                __syncwarp();
                for (int it = 0; it < p.J && it < 2; ++it) {
                    const int dg = p.diag(it);
                    if (dg < 0) continue;
                    const int s = (u0 + 2 * it + 1) % S::SLOTS, rows = min(ROWS, t.len - (p.J - 1 - it) * ROWS);
                    wait(raw(s), (rp >> s) & 1u);
                    rp ^= 1u << s;
                    unsigned char *v = smem + S::RING + s * S::TILE;
                    // x * 0 is zero unless x is not finite: one packed product a word, summed up
                    uint32_t acc[4] = {0, 0, 0, 0};
#pragma unroll 4
                    for (int i = lane; i < ROWS * 8; i += 32)
#pragma unroll
                        for (int c = 0; c < DP / 64; ++c) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(v + c * PANEL + i * 16);
                            acc[0] = fma_zero(x.x, acc[0]);
                            acc[1] = fma_zero(x.y, acc[1]);
                            acc[2] = fma_zero(x.z, acc[2]);
                            acc[3] = fma_zero(x.w, acc[3]);
                        }
                    if (__any_sync(FULL_MASK, (acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu)) {  // some row is not finite (or behind the document)
                        for (int r0 = 0; r0 < rows; r0 += 4) {       // 8 lanes a row
                            const int r = r0 + (lane >> 3);
                            bool x = false;
                            if (r < rows)
#pragma unroll
                                for (int c = 0; c < DP / 64; ++c)
                                    x |= any_nonfinite(*reinterpret_cast<const uint4 *>(v + c * PANEL + r * 128 + (lane & 7) * 16));
                            const uint32_t m = __ballot_sync(FULL_MASK, x);
                            for (int e = 0; e < 4; ++e)
                                if ((m >> (8 * e)) & 0xffu) {
                                    if (lane == 0) rows_bad[dg * 4 + ((r0 + e) >> 5)] |= 1u << ((r0 + e) & 31);
                                    if (lane < 8)
#pragma unroll
                                        for (int c = 0; c < DP / 64; ++c)
                                            *reinterpret_cast<uint4 *>(v + c * PANEL + (r0 + e) * 128 + lane * 16) = make_uint4(0, 0, 0, 0);
                                }
                        }
                    }
                    if (rows < ROWS) zero_tail<DP>(v, rows, lane);
                    __threadfence_block();
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(full(s));
                }
                feed.done(k, lane);
                u0 += 2 * p.J;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int i = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float c2 = a.scale * LOG2E, slack = HEADROOM / c2;
        const int64_t os = (int64_t)a.Hq * a.d;
        uint32_t sp = 0, op = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            if (t.h < 0) break;
            const Plan p = plan(t);
            if (t.len < 0) {  // rows that no document holds
                const int nh = pair_heads ? 2 : 1, nv = a.d / 8;
                for (int e = tid; e < -t.len * nh * nv; e += 256) {
                    const int r = e / (nh * nv), c = e % (nh * nv);
                    st16(static_cast<bf16 *>(a.o) + (t.start + r) * os + (int64_t)p.h0 * a.d + c * 8, make_uint4(0, 0, 0, 0));
                }
                for (int e = tid; e < -t.len * nh; e += 256) a.lse[(p.h0 + e % nh) * a.T + t.start + e / nh] = -INFINITY;
                feed.done(k, lane);
                continue;
            }
            const int steps = p.n[i];
            float m = 0.f, l = 0.f;
            for (int it = 0; it < steps; ++it) {
                wait(sfull(i), sp);
                sp ^= 1u;
                __syncwarp();
                tc::fence_after_sync();
                const u64 c2p = mk2(c2, c2);
                u64 sum[2] = {0, 0};
                auto half_there = [&] {  // P's first SPLIT columns are written
                    tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(phalf(i));
                };
                // 32 columns of P from S: the exponentials, their sum, bf16
                auto weights = [&](const float *s, u64 off, int c) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const u64 x = fma2(mk2(s[2 * e], s[2 * e + 1]), c2p, off);
                        const u64 y = mk2(ex2(lo2(x)), ex2(hi2(x)));
                        sum[e & 1] = add2(sum[e & 1], y);
                        w[e] = pack_bf2(lo2(y), hi2(y));
                    }
                    tmem_st16(tS[i] + lanes + c / 2, w);
                };
                if (it == 0) {
                    // The diagonal: this warp's rows see none of the 32-column blocks behind the warp's own, and part
                    // of that.  Two short passes over S, block by block, instead of 128 columns at once: code of its
                    // own that is little and skips what is masked.
                    float top = -INFINITY;
#pragma unroll 1
                    for (int b = 0; b <= quarter; ++b) {
                        float s[32];
                        tmem_ld32(tS[i] + lanes + 32 * b, s);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) top = fmaxf(top, b == quarter && c > lane ? -INFINITY : s[c]);
                    }
                    m = top == -INFINITY ? -1e30f : top;
                    const u64 off = mk2(fmaf(-m, c2, -HEADROOM), fmaf(-m, c2, -HEADROOM));
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        if (b <= quarter) {
                            float s[32];
                            tmem_ld32(tS[i] + lanes + 32 * b, s);
                            tc::tmem_wait_ld();
                            if (b == quarter) {
#pragma unroll
                                for (int c = 0; c < 32; ++c) s[c] = c > lane ? -INFINITY : s[c];
                            }
                            weights(s, off, 32 * b);
                        } else {
                            const uint32_t zero[16] = {};
                            tmem_st16(tS[i] + lanes + 16 * b, zero);
                        }
                        if (32 * b + 32 == SPLIT) half_there();
                    }
                } else {
                    float s[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(tS[i] + lanes + 32 * c, s + 32 * c);
                    tc::tmem_wait_ld();
                    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int c = 4; c < 124; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + e], s[c + 4 + e]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[124 + e]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (__any_sync(FULL_MASK, top > m + slack)) {
                        const float mn = top > m + slack ? top : m, f = ex2((m - mn) * c2);  // other rows keep theirs (f = 1)
                        l *= f;
                        m = mn;
#pragma unroll 1
                        for (int c = 0; c < DP; c += 8) {  // seldom: few registers rather than few turns
                            float o[8];
                            tc::tmem_ld8(tO[i] + lanes + c, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] *= f;
                            tmem_st8(tO[i] + lanes + c, o);
                        }
                    }
                    const u64 off = mk2(fmaf(-m, c2, -HEADROOM), fmaf(-m, c2, -HEADROOM));
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        weights(s + c, off, c);
                        if (c + 32 == SPLIT) half_there();
                    }
                }
                const u64 both = add2(sum[0], sum[1]);
                l += lo2(both) + hi2(both);
                tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(pfull(i));
            }
            if (steps) {  // o = O / l, lse = m scale + log(2^16 l)
                wait(ofull(i), op);
                op ^= 1u;
                __syncwarp();
                tc::fence_after_sync();
                const int r = t.r0 + (pair_heads ? 0 : i * ROWS) + row, h = pair_heads ? p.h0 + i : p.h0;
                const int64_t at = (int64_t)t.start + r;
                const float inv = 1.f / l, lse = m * a.scale + (logf(l) + HEADROOM * LN2);
                const bool on = r < t.len;
                if (on) a.lse[h * a.T + at] = lse;
                // The value rows kept out of the products that this tile took part in: its own diagonal's, of which a row
                // sees those up to itself, and for the second of two tiles of one head also the first one's diagonal, of
                // which it sees all.
                const int own = pair_heads ? 0 : i;
                for (int g = 0; g <= own; ++g) {
                    const volatile uint32_t *mask = bad + (k % FEED_SLOTS) * 8 + g * 4;
                    if (mask[0] | mask[1] | mask[2] | mask[3])
                        add_rows(a, tO[i] + lanes, static_cast<const bf16 *>(a.q) + at * a.qs + (int64_t)h * a.d, h / a.group,
                                 at - row - (own - g) * ROWS, !on ? -1 : (g < own ? ROWS - 1 : row), c2,
                                 fmaf(-m, c2, -HEADROOM), mask);
                }
                bf16 *o = static_cast<bf16 *>(a.o) + (at - lane) * os + (int64_t)h * a.d;  // the warp's first row
                const int left = t.len - (r - lane);                                       // its rows inside the document
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {  // not unrolled: this code runs once an item, from a cold cache
                    float x[32];
                    tmem_ld32(tO[i] + lanes + c, x);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] *= inv;
                    if (c < a.d) store_rows32(o + c, os, x, left, a.d - c, lane);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(oempty(i));
            }
            feed.done(k, lane);
        }
    }

    // The loading and the issuing warp have waited for their own copies and products.
    if (timed_out) atomicExch(&g_dsc_status_attn_fwd, (int)DSC_ERR_TIMEOUT);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// A feed whose waits run out: warp 1 reads item 0, which nothing puts there, and
// warp 0 draws an item for a slot that nothing empties.  Both must end the feed,
// and the slot keeps what it held; anything else is reported as an error of its
// own.
__global__ void k_feed_selftest(long long limit) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Feed feed(tc::smem_u32(smem), smem, 0);
    int32_t cu[2] = {0, 0};
    AttnArgs a{};
    a.cu = cu;  // a list made here; its documents are not read
    if (tid == 0) {
        feed.init(1);
        for (int i = 0; i < FEED_SLOTS; ++i) feed.items[i] = Item{1 << 29, 1 << 29, 0, 7};
        *feed.head = INLINE_TILES;
        for (int i = 0; i < INLINE_TILES; ++i) feed.tiles()[i] = AttnTile{0, 1, 0, 0};
        tc::fence_mbar_init();
    }
    __syncthreads();
    bool timed_out = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!timed_out && !tc::mbar_wait(bar, parity, limit)) timed_out = true;
    };
    int h = -1;
    if (warp == 1) h = feed.get(0, wait, timed_out).h;
    else if (lane == 0) h = feed.draw(FEED_SLOTS, a, 1, wait, timed_out).h;
    const bool part = tid == 0 || warp == 1, ok = h < 0 && timed_out && feed.items[0].h == 7;
    if (part && ok) atomicExch(&g_dsc_status_attn_fwd, (int)DSC_ERR_TIMEOUT);
    __syncthreads();
    if (part && !ok) atomicExch(&g_dsc_status_attn_fwd, (int)DSC_ERR_CUDA);
}

template <int DP> cudaError_t launch(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(k_attn_fwd_tc<DP>, Fwd<DP>::TOTAL, ready);
    if (e != cudaSuccess) return e;
    FwdMaps m;
    if (!rows_map(&m.q, a.q, a.T, a.Hq, a.d, a.qs) || !rows_map(&m.k, a.k, a.T, a.Hkv, a.d, a.ks) ||
        !rows_map(&m.v, a.v, a.T, a.Hkv, a.d, a.vs))
        return cudaErrorNotSupported;
    const int pair = a.group % 2 == 0, heads = pair ? a.Hq / 2 : a.Hq;
    const int64_t items = max_tiles * heads, blocks = items < c.sms ? items : c.sms;
    return launch_pdl(k_attn_fwd_tc<DP>, dim3((unsigned)blocks), dim3(THREADS), Fwd<DP>::TOTAL, c.stream, m, a,
                      heads, pair);
}

int take(cudaStream_t stream) {
    int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_dsc_status_attn_fwd, sizeof v, 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -1;
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_dsc_status_attn_fwd, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -1;
    return cudaStreamSynchronize(stream) == cudaSuccess ? v : -1;
}

}  // namespace
}  // namespace attn_tc

int attn_fwd_tc_rows(int group) { return group % 2 == 0 ? attn_tc::ROWS : 2 * attn_tc::ROWS; }

cudaError_t launch_attn_fwd_tc(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    return a.d <= 64 ? attn_tc::launch<64>(c, a, max_tiles) : attn_tc::launch<128>(c, a, max_tiles);
}

int take_attn_fwd_status(cudaStream_t stream) { return attn_tc::take(stream); }

cudaError_t launch_feed_selftest(cudaStream_t stream) {
    attn_tc::k_feed_selftest<<<1, 64, attn_tc::Feed::BYTES, stream>>>(10000000ll);
    count_launch();
    return cudaGetLastError();
}

}  // namespace dsc
