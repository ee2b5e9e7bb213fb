// Gradients of causal attention over packed documents on the tensor cores (bf16).
//
// Two kernels, each the sole owner of what it writes, so nothing depends on the
// order in which blocks run:
//
//   k_attn_dkv_tc  a block owns 128 keys of one key head and walks the query
//                  tiles that see them, for each query head of the group:
//                    S^T = K Q^T,  P^T = 2^(S^T c - lse),     dv += P^T dout
//                    dP^T = V dout^T,  dS^T = P^T (dP^T - D),  dk += dS^T Q
//   k_attn_dq_tc   a block owns 128 query rows of one head and walks their keys:
//                    S = Q K^T,  dP = dout V^T,  dS = P (dP - D),  dq += dS K
//
// Recomputing S and dP in the second kernel costs 2 of 7 products; the
// alternative, adding dq up in memory from the first, needs 32-bit atomics
// whose order would change the result.
//
// D_i = dout_i . o_i = sum_j P_ij dP_ij is summed up from P and dP in fp32, by the
// dq kernel, which runs first and leaves it to the other.  (From the o that the
// caller has, rounded to bf16, it would be off by 2^-9 |dout| |o|, which can be
// all that remains of dP - D where few keys carry a row: dq was then 1.5 to 1.9
// times as far off as the products' own roundings leave it.)  An item of N key
// tiles takes 2 N - 1 steps: the sums over the tiles before the diagonal, the
// diagonal's sum and at once its gradient, and the gradient of the others from
// there back.  5 products a pair of tiles instead of 3, and no pass over o: the
// gradients of 16384 tokens in 23 documents, 16 heads of 128, take 299 us
// against 283 with a D from o, of one document of 8192, 32/8 heads, 1887
// against 1471 (the added steps' K and V come from L2 at 9 TB/s, which bounds them).
//
// Roles as in the forward: warps 0-7 do the elementwise part (a thread owns a
// row of the 128 x 128 tile and 64 of its columns; P^T and dS^T go back to
// tensor memory as bf16 and are the A operand of the accumulating products),
// warp 8 loads, warp 9 issues the products, warp 10 keeps the row statistics
// coming and zeroes operand rows that lie behind the document (their weights
// are zero, and 0 * NaN would reach the sums), warps 12-15 write the finished
// gradients (done by the elementwise warps, that took 3500 of an item's cycles
// between its last and the next one's first step).
//
// Blocks are persistent: an item's first products run under the previous one's
// epilogue.  Order of the products, so that the tensor cores work while the elementwise
// warps do (step u of dk/dv):   ... | dv(u), S(u+1) | dk(u), dP(u+1) | ...
//                                     | dS(u) formed | P(u+1) formed  |
// (heads of 64: S(u+2), into the second of two buffers, in the place of S(u+1))
// and of dq, with two S buffers: ... | dP(j+1), dq(j), S(j+2) | ... (dq(j) from the diagonal on)
#include "attn_tc.cuh"

namespace dsc {
namespace attn_tc {

__device__ int g_dsc_status_attn_bwd = 0;

namespace {

constexpr int THREADS = 512;
// Registers a thread: launched with 128 (all 65536 of the SM), then dealt out
// per warpgroup (256 * 168 + 128 * 80 + 128 * 96 = 65536).
constexpr int REGS_ELEM = 168, REGS_OTHER = 80, REGS_OUT = 96;

struct BwdMaps {
    CUtensorMap q, k, v, dout;
};

// Four probabilities 2^(S c + n) in place.  With heads of 64 the products are
// short and the exponential unit's 16 results a cycle and SM hold a step up, so
// every other pair goes to the FMA pipe (5003 tokens, 14/2 heads: gradients 86 us
// against 94); with 128 the exponentials run under the products (8192 tokens,
// 32/8 heads: 1943 us against 1972 with half of them there).
template <int DP> __device__ __forceinline__ void weights4(float *s, u64 c, u64 n0, u64 n1) {
    const u64 x = fma2(mk2(s[0], s[1]), c, n0), z = fma2(mk2(s[2], s[3]), c, n1);
    s[0] = ex2(lo2(x));
    s[1] = ex2(hi2(x));
    const u64 y = DP == 64 ? ex2_fma(z) : mk2(ex2(lo2(z)), ex2(hi2(z)));
    s[2] = lo2(y);
    s[3] = hi2(y);
}
// x = p (x + n), a pair
__device__ __forceinline__ void times2(float *x, const float *p, u64 n) {
    const u64 y = mul2(mk2(p[0], p[1]), add2(mk2(x[0], x[1]), n));
    x[0] = lo2(y);
    x[1] = hi2(y);
}

// N columns of a warp's 32 accumulator rows times f, as bf16, from row 0 and column 0 at g (rows < n, columns < ncol).
template <int N> __device__ __forceinline__ void store_acc(bf16 *g, int64_t stride, uint32_t taddr, float f, int n, int ncol, int lane) {
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {  // not unrolled: this code runs once an item, from a cold cache
        float x[32];
        tmem_ld32(taddr + c, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] *= f;
        if (c < ncol) store_rows32(g + c, stride, x, n, ncol - c, lane);
    }
}

// N columns of an accumulator row as they are, to global memory in fp32 (columns < d).
template <int N> __device__ __forceinline__ void store_part(float *g, uint32_t taddr, int d, bool on) {
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        float x[32];
        tmem_ld32(taddr + c, x);
        tc::tmem_wait_ld();
        if (on)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                if (c + e >= d) break;
                const float y[4] = {x[e], x[e + 1], x[e + 2], x[e + 3]};
                st16(g + c + e, pack(y));
            }
    }
}

// Rows of one head to zero, by the 256 elementwise threads.
template <typename T> __device__ __forceinline__ void zero_head(T *g, int64_t stride, int rows, int d, int tid) {
    constexpr int V = VecOf<T>::V;
    const int nv = d / V;
    for (int i = tid; i < rows * nv; i += 256) st16(g + (i / nv) * stride + (i % nv) * V, make_uint4(0, 0, 0, 0));
}

// ------------------------------------------------------------- dk, dv ---

template <int DP> struct Dkv {
    static constexpr uint32_t TILE = PANEL * (DP / 64);
    // S is formed NS steps ahead: with two buffers (heads of 64 leave room in
    // tensor memory) P(u+1) does not wait for the products that P(u) goes into.
    static constexpr int NS = DP == 64 ? 2 : 1;
    static constexpr int STAGES = DP == 64 ? 4 : 2;        // of Q, dout
    static constexpr uint32_t RING = 2 * TILE;             // after K, V
    static constexpr uint32_t STATS = RING + STAGES * 2 * TILE;  // two stages of (-lse log2 e, -D), 128 each
    static constexpr uint32_t BARS = STATS + 2 * 1024;
    static constexpr uint32_t FEED = BARS + 256;
    // tensor memory: S buffers, dP, dv, dk
    static constexpr uint32_t TP = NS * 128, TV = TP + 128, TK = TV + DP;
    // more than a third of the shared memory, so that one block has the SM's tensor memory
    static constexpr uint32_t USED = FEED + Feed::BYTES + 16 + 1024;
    static constexpr uint32_t TOTAL = USED < 120 * 1024 ? 120 * 1024 : USED;
};

// An item is (key tile, key head, part of the head's query heads): `heads` = Hkv * nsplit.
template <int DP>
__global__ void __launch_bounds__(THREADS, 1)
    k_attn_dkv_tc(const __grid_constant__ BwdMaps maps, const __grid_constant__ AttnArgs a, int heads) {
    using S = Dkv<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = sbase + S::BARS;
    const uint32_t kvfull = bars, kvempty = bars + 8, dpfull = bars + 16, dsfull = bars + 24;
    const uint32_t vaccfull = bars + 32, kaccfull = bars + 40, vaccempty = bars + 48, kaccempty = bars + 56;
    auto full = [&](int g) { return bars + 64u + 8u * (uint32_t)(g % S::STAGES); };
    auto empty = [&](int g) { return bars + 96u + 8u * (uint32_t)(g % S::STAGES); };
    auto raw = [&](int g) { return bars + 128u + 8u * (uint32_t)(g % S::STAGES); };
    auto stfull = [&](int g) { return bars + 160u + 8u * (uint32_t)(g & 1); };
    auto stempty = [&](int g) { return bars + 176u + 8u * (uint32_t)(g & 1); };
    auto sfull = [&](int g) { return bars + 192u + 8u * (uint32_t)(g % S::NS); };
    auto pfull = [&](int g) { return bars + 208u + 8u * (uint32_t)(g % S::NS); };
    const Feed feed(sbase, smem, S::FEED);

    if (tid == 0) {
        tc::mbar_init(kvfull, 1);
        tc::mbar_init(kvempty, 1);
        tc::mbar_init(dpfull, 1);
        tc::mbar_init(dsfull, 8);
        tc::mbar_init(vaccfull, 1);
        tc::mbar_init(kaccfull, 1);
        tc::mbar_init(vaccempty, 4);
        tc::mbar_init(kaccempty, 4);
        for (int g = 0; g < S::STAGES; ++g) {
            tc::mbar_init(full(g), 1);
            tc::mbar_init(empty(g), 1);
            tc::mbar_init(raw(g), 1);
        }
        for (int g = 0; g < 2; ++g) {
            tc::mbar_init(stfull(g), 1);
            tc::mbar_init(stempty(g), 8);
        }
        for (int g = 0; g < S::NS; ++g) {
            tc::mbar_init(sfull(g), 1);
            tc::mbar_init(pfull(g), 8);
        }
        feed.init(14);  // all warps but the loading and the idle one
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&maps.q);
        tc::tma_prefetch_desc(&maps.k);
        tc::tma_prefetch_desc(&maps.v);
        tc::tma_prefetch_desc(&maps.dout);
    }
    if (warp == 9) {
        tc::tmem_alloc(sbase + S::FEED + Feed::BYTES, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = 0;  // the whole of the tensor memory: the allocation can only start at column 0
    const uint32_t tP = tmem + S::TP, tV = tmem + S::TV, tK = tmem + S::TK;
    auto tS = [&](int g) { return tmem + 128u * (uint32_t)(g % S::NS); };
    pdl_wait();
    pdl_trigger();
    feed.make_list(a, ROWS, true, tid);

    const long long limit = wait_limit(a);
    bool timed_out = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!timed_out && !tc::mbar_wait(bar, parity, limit)) timed_out = true;
    };
    // Steps of an item: query tile u % nqt (from the diagonal on) of query head h0 + u / nqt.
    struct Plan {
        int hk, sp, h0;      // key head, part, first query head
        int row0;            // first key; the query tiles start there too
        int rest, nqt, tail; // rows from there on, tiles of them, rows of the last one (0: all)
        int N;               // steps
        __device__ bool partial(int u) const { return tail && u % nqt == nqt - 1; }
    };
    const int gs = a.group / a.nsplit;
    auto plan = [&](const Item &t) {
        Plan p;
        p.hk = t.h / a.nsplit;
        p.sp = t.h % a.nsplit;
        p.h0 = p.hk * a.group + p.sp * gs;
        p.row0 = t.start + t.r0;
        p.rest = t.len - t.r0;
        p.nqt = (p.rest + ROWS - 1) / ROWS;
        p.tail = p.rest & (ROWS - 1);
        p.N = p.nqt * gs;
        return p;
    };
    auto stage = [&](int g) { return sbase + S::RING + (uint32_t)(g % S::STAGES) * 2 * S::TILE; };

    if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == 8) {
        if (lane == 0) {
            int g = 0, uses = 0;  // steps and items so far
            for (int k = 0;; ++k) {
                const Item t = feed.draw(k, a, heads, wait, timed_out);
                if (t.h < 0) break;
                if (t.len < 0) continue;
                const Plan p = plan(t);
                if (uses) wait(kvempty, (uint32_t)((uses - 1) & 1));
                if (timed_out) break;
                ++uses;
                tc::mbar_expect_tx(kvfull, 2 * S::TILE);
                load_rows<DP>(sbase, &maps.k, p.hk, p.row0, kvfull);
                load_rows<DP>(sbase + S::TILE, &maps.v, p.hk, p.row0, kvfull);
                for (int u = 0; u < p.N; ++u, ++g) {
                    if (g >= S::STAGES) wait(empty(g), (uint32_t)((g / S::STAGES - 1) & 1));
                    if (timed_out) break;
                    const uint32_t bar = p.partial(u) ? raw(g) : full(g);
                    const int h = p.h0 + u / p.nqt, r = p.row0 + (u % p.nqt) * ROWS;
                    tc::mbar_expect_tx(bar, 2 * S::TILE);
                    load_rows<DP>(stage(g), &maps.q, h, r, bar);
                    load_rows<DP>(stage(g) + S::TILE, &maps.dout, h, r, bar);
                }
            }
            // every load has landed before the block may end
            if (uses) tc::mbar_wait(kvfull, (uint32_t)((uses - 1) & 1), limit);
            for (int s = 0; s < S::STAGES && s < g; ++s) {
                const int last = s + ((g - 1 - s) / S::STAGES) * S::STAGES;
                tc::mbar_wait(full(s), (uint32_t)((last / S::STAGES) & 1), limit);
            }
        }
    } else if (warp == 9) {
        int g0 = 0, uses = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            if (t.len < 0) continue;
            const Plan p = plan(t);
            auto scores = [&](int u) {
                const int g = g0 + u;
                wait(full(g), (uint32_t)((g / S::STAGES) & 1));
                tc::fence_after_sync();
                mma_tiles<DP>(tS(g), sbase, stage(g));
                commit(sfull(g));
            };
            auto weights = [&](int u) {  // dP
                mma_tiles<DP>(tP, sbase + S::TILE, stage(g0 + u) + S::TILE);
                commit(dpfull);
                if (u + 1 == p.N) commit(kvempty);  // the scores were all issued before
            };
            wait(kvfull, (uint32_t)(uses & 1));
            scores(0);
            weights(0);
            if (S::NS == 2 && p.N > 1) scores(1);
            for (int u = 0; u < p.N; ++u) {
                const int g = g0 + u;
                if (u == 0 && uses) wait(vaccempty, (uint32_t)((uses - 1) & 1));
                wait(pfull(g), (uint32_t)((g / S::NS) & 1));
                tc::fence_after_sync();
                mma_rows<DP, 0, ROWS / 16, true>(tV, tS(g), stage(g) + S::TILE, u > 0);
                if (u + 1 == p.N) commit(vaccfull);
                if (u + S::NS < p.N) scores(u + S::NS);
                if (u == 0 && uses) wait(kaccempty, (uint32_t)((uses - 1) & 1));
                wait(dsfull, (uint32_t)(g & 1));
                tc::fence_after_sync();
                mma_rows<DP, 0, ROWS / 16, true>(tK, tP, stage(g), u > 0);
                commit(empty(g));
                if (u + 1 < p.N) weights(u + 1);
            }
            commit(kaccfull);
            g0 += p.N;
            ++uses;
        }
        if (uses) tc::mbar_wait(kaccfull, (uint32_t)((uses - 1) & 1), limit);  // every product is done
    } else if (warp == 10) {
        int g = 0;
        uint32_t rp = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            if (t.len < 0) continue;
            const Plan p = plan(t);
            for (int u = 0; u < p.N; ++u, ++g) {
                const int b = g & 1, h = p.h0 + u / p.nqt, q0 = (u % p.nqt) * ROWS;
                float x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = q0 + lane + 32 * i;
                    const int64_t at = h * a.T + p.row0 + r;
                    x[i] = r < p.rest ? -a.lse[at] * LOG2E : -INFINITY;
                    y[i] = r < p.rest ? -a.delta[at] : 0.f;
                }
                if (g >= 2) wait(stempty(g), (uint32_t)((g / 2 - 1) & 1));
                float *st = reinterpret_cast<float *>(smem + S::STATS + b * 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    st[lane + 32 * i] = x[i];
                    st[128 + lane + 32 * i] = y[i];
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(stfull(g));
                if (p.partial(u)) {
                    const int s = g % S::STAGES;
                    wait(raw(g), (rp >> s) & 1u);
                    rp ^= 1u << s;
                    unsigned char *q = smem + (stage(g) - sbase);
                    zero_tail<DP>(q, p.tail, lane);
                    zero_tail<DP>(q + S::TILE, p.tail, lane);
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(full(g));
                }
            }
        }
    }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ELEM));
        const int half = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, c0 = 64 * half;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float c2 = a.scale * LOG2E;
        int g = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            const Plan p = plan(t);
            const int64_t ps = (int64_t)a.Hkv * a.d;
            if (t.len < 0) {
                if (a.nsplit > 1) {
                    zero_head(a.kpart + ((int64_t)p.sp * a.T * a.Hkv + p.hk) * a.d + t.start * ps, ps, -t.len, a.d, tid);
                    zero_head(a.vpart + ((int64_t)p.sp * a.T * a.Hkv + p.hk) * a.d + t.start * ps, ps, -t.len, a.d, tid);
                } else {
                    zero_head(static_cast<bf16 *>(a.dk) + (int64_t)p.hk * a.d + t.start * a.dks, a.dks, -t.len, a.d, tid);
                    zero_head(static_cast<bf16 *>(a.dv) + (int64_t)p.hk * a.d + t.start * a.dvs, a.dvs, -t.len, a.d, tid);
                }
                continue;
            }
            for (int u = 0; u < p.N; ++u, ++g) {
                const int b = g & 1;
                const bool diag = u % p.nqt == 0;
                const float4 *nl = reinterpret_cast<const float4 *>(smem + S::STATS + b * 1024) + c0 / 4, *nd = nl + 32;
                float w[64];
                wait(stfull(g), (uint32_t)((g >> 1) & 1));
                wait(sfull(g), (uint32_t)((g / S::NS) & 1));
                __syncwarp();
                tc::fence_after_sync();
                tmem_ld32(tS(g) + lanes + c0, w);
                tmem_ld32(tS(g) + lanes + c0 + 32, w + 32);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 n = nl[c / 4];
                    weights4<DP>(w + c, mk2(c2, c2), mk2(n.x, n.y), mk2(n.z, n.w));
                }
                if (diag) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) w[c] = c0 + c < row ? 0.f : w[c];
                }
                uint32_t z[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) z[c] = pack_bf2(w[2 * c], w[2 * c + 1]);
                tmem_st32(tS(g) + lanes + c0, z);
                tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(pfull(g));

                wait(dpfull, (uint32_t)(g & 1));
                __syncwarp();
                tc::fence_after_sync();
#pragma unroll
                for (int e = 0; e < 64; e += 32) {
                    float x[32];
                    tmem_ld32(tP + lanes + c0 + e, x);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 n = nd[(e + c) / 4];
                        times2(x + c, w + e + c, mk2(n.x, n.y));
                        times2(x + c + 2, w + e + c + 2, mk2(n.z, n.w));
                    }
                    if (diag) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = c0 + e + c < row ? 0.f : x[c];
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) z[e / 2 + c] = pack_bf2(x[2 * c], x[2 * c + 1]);
                }
                tmem_st32(tP + lanes + c0, z);
                tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(dsfull);
                    tc::mbar_arrive(stempty(g));
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OUT));
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        int uses = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            if (t.len < 0) continue;
            const Plan p = plan(t);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {  // dv, then dk
                wait(half ? kaccfull : vaccfull, (uint32_t)(uses & 1));
                __syncwarp();
                tc::fence_after_sync();
                const int64_t r = (int64_t)p.row0 + row;
                const uint32_t acc = (half ? tK : tV) + lanes;
                if (a.nsplit > 1) {
                    float *part = (half ? a.kpart : a.vpart) + ((int64_t)p.sp * a.T * a.Hkv + p.hk) * a.d;
                    store_part<DP>(part + r * a.Hkv * a.d, acc, a.d, row < p.rest);
                } else {
                    const int64_t outs = half ? a.dks : a.dvs;
                    bf16 *out = static_cast<bf16 *>(half ? a.dk : a.dv) + (int64_t)p.hk * a.d + (r - lane) * outs;
                    store_acc<DP>(out, outs, acc, half ? a.scale : 1.f, p.rest - quarter * 32, a.d, lane);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(half ? kaccempty : vaccempty);
            }
            ++uses;
        }
    }

    // The loading and the issuing warp have waited for their own copies and products.
    if (timed_out) atomicExch(&g_dsc_status_attn_bwd, (int)DSC_ERR_TIMEOUT);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ----------------------------------------------------------------- dq ---

template <int DP> struct Dq {
    static constexpr uint32_t TILE = PANEL * (DP / 64);
    static constexpr int KS = 3, VS = 2;                   // ring slots
    static constexpr uint32_t KRING = 2 * TILE;            // after Q and dout
    static constexpr uint32_t VRING = KRING + KS * TILE;
    static constexpr uint32_t BARS = VRING + VS * TILE;
    static constexpr uint32_t SUMS = BARS + 192;           // [2][128]: each half's sum over a row's columns
    static constexpr uint32_t FEED = SUMS + 1024;
    // nothing over for alignment: without static shared memory the dynamic begins at a multiple of 1024
    static constexpr uint32_t USED = FEED + Feed::BYTES + 16;
    static constexpr uint32_t TOTAL = USED < 120 * 1024 ? 120 * 1024 : USED;
};

template <int DP>
__global__ void __launch_bounds__(THREADS, 1)
    k_attn_dq_tc(const __grid_constant__ BwdMaps maps, const __grid_constant__ AttnArgs a, int heads) {
    using S = Dq<DP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = tc::smem_u32(smem);
    if (sbase & 1023u) {  // the tiles' swizzle would be off: never so far, and reported if it ever is
        atomicExch(&g_dsc_status_attn_bwd, (int)DSC_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = sbase + S::BARS;
    const uint32_t qfull = bars, dpfull = bars + 8, dsfull = bars + 16, accfull = bars + 24, qempty = bars + 32, accempty = bars + 40;
    auto sfull = [&](int s) { return bars + 48u + 8u * (uint32_t)s; };
    auto kfull = [&](int s) { return bars + 64u + 8u * (uint32_t)s; };
    auto kempty = [&](int s) { return bars + 88u + 8u * (uint32_t)s; };
    auto kraw = [&](int s) { return bars + 112u + 8u * (uint32_t)s; };
    auto vfull = [&](int s) { return bars + 136u + 8u * (uint32_t)s; };
    auto vempty = [&](int s) { return bars + 152u + 8u * (uint32_t)s; };
    const uint32_t sumfull = bars + 168, sumread = bars + 176;
    const Feed feed(sbase, smem, S::FEED);
    float *sums = reinterpret_cast<float *>(smem + S::SUMS);

    if (tid == 0) {
        tc::mbar_init(qfull, 1);
        tc::mbar_init(qempty, 1);
        tc::mbar_init(dpfull, 1);
        tc::mbar_init(dsfull, 8);
        tc::mbar_init(accfull, 1);
        tc::mbar_init(accempty, 4);
        tc::mbar_init(sumfull, 8);
        tc::mbar_init(sumread, 8);
        for (int s = 0; s < 2; ++s) tc::mbar_init(sfull(s), 1);
        for (int s = 0; s < S::KS; ++s) {
            tc::mbar_init(kfull(s), 1);
            tc::mbar_init(kempty(s), 1);
            tc::mbar_init(kraw(s), 1);
        }
        for (int s = 0; s < S::VS; ++s) {
            tc::mbar_init(vfull(s), 1);
            tc::mbar_init(vempty(s), 1);
        }
        feed.init(14);  // all warps but the loading and the idle one
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&maps.q);
        tc::tma_prefetch_desc(&maps.k);
        tc::tma_prefetch_desc(&maps.v);
        tc::tma_prefetch_desc(&maps.dout);
    }
    if (warp == 9) {
        tc::tmem_alloc(sbase + S::FEED + Feed::BYTES, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = 0;  // the whole of the tensor memory: the allocation can only start at column 0
    const uint32_t tS = tmem, tP = tmem + 256, tQ = tmem + 384;  // tS: two buffers
    pdl_wait();
    pdl_trigger();
    feed.make_list(a, ROWS, false, tid);

    const long long limit = wait_limit(a);
    bool timed_out = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!timed_out && !tc::mbar_wait(bar, parity, limit)) timed_out = true;
    };
    auto kslot = [&](int g) { return sbase + S::KRING + (uint32_t)(g % S::KS) * S::TILE; };
    auto vslot = [&](int g) { return sbase + S::VRING + (uint32_t)(g % S::VS) * S::TILE; };
    // An item: N key tiles in 2 N - 1 steps, up to the diagonal (step N - 1) and back; `rows` rows of the query tile, and
    // keys of the diagonal's tile.
    auto tiles = [](const Item &t) { return t.r0 / ROWS + 1; };
    auto rows_of = [](const Item &t) { return min(ROWS, t.len - t.r0); };

    if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == 8) {
        if (lane == 0) {
            int g = 0, gk = 0, uses = 0;  // steps, K tiles loaded and items so far
            for (int k = 0;; ++k) {
                const Item t = feed.draw(k, a, heads, wait, timed_out);
                if (t.h < 0) break;
                if (t.len < 0) continue;
                const int N = tiles(t), rows = rows_of(t), hk = t.h / a.group;
                if (uses) wait(qempty, (uint32_t)((uses - 1) & 1));
                if (timed_out) break;
                ++uses;
                tc::mbar_expect_tx(qfull, 2 * S::TILE);
                load_rows<DP>(sbase, &maps.q, t.h, t.start + t.r0, qfull);
                load_rows<DP>(sbase + S::TILE, &maps.dout, t.h, t.start + t.r0, qfull);
                for (int j = 0; j < 2 * N - 1; ++j, ++g) {
                    const int r = t.start + (j < N ? j : 2 * N - 2 - j) * ROWS, sk = g % S::KS, sv = g % S::VS;
                    if (g >= S::KS) wait(kempty(sk), (uint32_t)((g / S::KS - 1) & 1));
                    if (timed_out) break;
                    const uint32_t bar = j == N - 1 && rows < ROWS ? kraw(sk) : kfull(sk);
                    tc::mbar_expect_tx(bar, S::TILE);
                    load_rows<DP>(kslot(g), &maps.k, hk, r, bar);
                    gk = g + 1;
                    if (g >= S::VS) wait(vempty(sv), (uint32_t)((g / S::VS - 1) & 1));
                    if (timed_out) break;
                    tc::mbar_expect_tx(vfull(sv), S::TILE);
                    load_rows<DP>(vslot(g), &maps.v, hk, r, vfull(sv));
                }
            }
            // every load has landed before the block may end
            if (uses) tc::mbar_wait(qfull, (uint32_t)((uses - 1) & 1), limit);
            for (int s = 0; s < S::KS && s < gk; ++s) {
                const int last = s + ((gk - 1 - s) / S::KS) * S::KS;
                tc::mbar_wait(kfull(s), (uint32_t)((last / S::KS) & 1), limit);
            }
            for (int s = 0; s < S::VS && s < g; ++s) {
                const int last = s + ((g - 1 - s) / S::VS) * S::VS;
                tc::mbar_wait(vfull(s), (uint32_t)((last / S::VS) & 1), limit);
            }
        }
    } else if (warp == 9) {
        int g0 = 0, uses = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            if (t.len < 0) continue;
            const int first = tiles(t) - 1, M = 2 * first + 1;  // the first step with a gradient, steps
            auto scores = [&](int g) {
                wait(kfull(g % S::KS), (uint32_t)((g / S::KS) & 1));
                tc::fence_after_sync();
                mma_tiles<DP>(tS + 128u * (g & 1), sbase, kslot(g));
                commit(sfull(g & 1));
            };
            auto weights = [&](int g) {  // dP
                wait(vfull(g % S::VS), (uint32_t)((g / S::VS) & 1));
                tc::fence_after_sync();
                mma_tiles<DP>(tP, sbase + S::TILE, vslot(g));
                commit(dpfull);
                commit(vempty(g % S::VS));
            };
            wait(qfull, (uint32_t)(uses & 1));
            scores(g0);
            weights(g0);
            if (M > 1) scores(g0 + 1);
            else commit(qempty);
            for (int j = 0; j < M; ++j) {
                const int g = g0 + j;
                wait(dsfull, (uint32_t)(g & 1));
                tc::fence_after_sync();
                if (j + 1 < M) {
                    weights(g + 1);
                    if (j + 2 == M) commit(qempty);  // its scores were issued a step ago
                }
                if (j == first && uses) wait(accempty, (uint32_t)((uses - 1) & 1));
                if (j >= first) mma_rows<DP, 0, ROWS / 16, true>(tQ, tS + 128u * (g & 1), kslot(g), j > first);
                commit(kempty(g % S::KS));
                if (j + 2 < M) scores(g + 2);
            }
            commit(accfull);
            g0 += M;
            ++uses;
        }
        if (uses) tc::mbar_wait(accfull, (uint32_t)((uses - 1) & 1), limit);  // every product is done
    } else if (warp == 10) {
        int g = 0;
        uint32_t rp = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            if (t.len < 0) continue;
            const int rows = rows_of(t), first = tiles(t) - 1, s = (g + first) % S::KS;
            if (rows < ROWS) {
                wait(kraw(s), (rp >> s) & 1u);
                rp ^= 1u << s;
                zero_tail<DP>(smem + (kslot(g + first) - sbase), rows, lane);
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(kfull(s));
            }
            g += 2 * first + 1;
        }
    }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ELEM));
        const int half = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, c0 = 64 * half;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float c2 = a.scale * LOG2E;
        int g = 0, totals = 0;  // steps and row totals so far
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            bf16 *dq = static_cast<bf16 *>(a.dq) + (int64_t)t.h * a.d;
            if (t.len < 0) {
                zero_head(dq + t.start * a.dqs, a.dqs, -t.len, a.d, tid);
                continue;
            }
            const int first = tiles(t) - 1, M = 2 * first + 1;
            const int64_t r = (int64_t)t.start + t.r0 + row;
            const bool on = row < rows_of(t);
            const float nl = on ? -a.lse[t.h * a.T + r] * LOG2E : -INFINITY;
            float nd = 0.f;  // -D
            u64 sum[2] = {0, 0};  // of P dP, this half's columns
            // Sum over the row of both halves' `own`.  Bounded waits, not bar.sync: a warp whose wait has run out takes
            // no further item, and the others must not wait for it without end.
            auto row_total = [&](float own) {
                if (totals) wait(sumread, (uint32_t)((totals - 1) & 1));  // the last item's have been read
                __syncwarp();
                sums[half * ROWS + row] = own;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(sumfull);
                wait(sumfull, (uint32_t)(totals & 1));
                ++totals;
                const float v = sums[row] + sums[ROWS + row];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(sumread);
                return v;
            };
            for (int j = 0; j < M; ++j, ++g) {
                const uint32_t tb = tS + 128u * (g & 1) + lanes + c0;
                float w[64];
                wait(sfull(g & 1), (uint32_t)((g >> 1) & 1));
                __syncwarp();
                tc::fence_after_sync();
                tmem_ld32(tb, w);
                tmem_ld32(tb + 32, w + 32);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 64; c += 4) weights4<DP>(w + c, mk2(c2, c2), mk2(nl, nl), mk2(nl, nl));
                uint32_t z[32];
                wait(dpfull, (uint32_t)(g & 1));
                __syncwarp();
                tc::fence_after_sync();
                if (j <= first) {
#pragma unroll
                    for (int e = 0; e < 64; e += 32) {
                        float x[32];
                        tmem_ld32(tP + lanes + c0 + e, x);
                        tc::tmem_wait_ld();
                        if (j == first) {  // a masked pair counts for nothing, whatever it holds
#pragma unroll
                            for (int c = 0; c < 32; ++c) x[c] = c0 + e + c > row ? 0.f : x[c];
#pragma unroll
                            for (int c = 0; c < 32; ++c) w[e + c] = c0 + e + c > row ? 0.f : w[e + c];
                        }
#pragma unroll
                        for (int c = 0; c < 32; c += 2) sum[c >> 1 & 1] = fma2(mk2(w[e + c], w[e + c + 1]), mk2(x[c], x[c + 1]), sum[c >> 1 & 1]);
                    }
                    if (j < first) {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(dsfull);
                        continue;
                    }
                    const u64 both = add2(sum[0], sum[1]);
                    nd = -row_total(lo2(both) + hi2(both));
                }
#pragma unroll
                for (int e = 0; e < 64; e += 32) {
                    float x[32];
                    tmem_ld32(tP + lanes + c0 + e, x);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; c += 2) times2(x + c, w + e + c, mk2(nd, nd));
                    if (j == first) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = c0 + e + c > row ? 0.f : x[c];
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) z[e / 2 + c] = pack_bf2(x[2 * c], x[2 * c + 1]);
                }
                tmem_st32(tb, z);
                tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(dsfull);
            }
            if (half == 0 && on) a.delta[t.h * a.T + r] = -nd;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OUT));
        const int quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        int uses = 0;
        for (int k = 0;; ++k) {
            const Item t = feed.get(k, wait, timed_out);
            feed.done(k, lane);
            if (t.h < 0) break;
            if (t.len < 0) continue;
            wait(accfull, (uint32_t)(uses & 1));
            ++uses;
            __syncwarp();
            tc::fence_after_sync();
            bf16 *dq = static_cast<bf16 *>(a.dq) + (int64_t)t.h * a.d + ((int64_t)t.start + t.r0 + quarter * 32) * a.dqs;
            store_acc<DP>(dq, a.dqs, tQ + lanes, a.scale, rows_of(t) - quarter * 32, a.d, lane);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(accempty);
        }
    }

    if (timed_out) atomicExch(&g_dsc_status_attn_bwd, (int)DSC_ERR_TIMEOUT);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

bool bwd_maps(const AttnArgs &a, BwdMaps &m) {
    return rows_map(&m.q, a.q, a.T, a.Hq, a.d, a.qs) && rows_map(&m.k, a.k, a.T, a.Hkv, a.d, a.ks) &&
           rows_map(&m.v, a.v, a.T, a.Hkv, a.d, a.vs) && rows_map(&m.dout, a.dout, a.T, a.Hq, a.d, (int64_t)a.Hq * a.d);
}

template <auto kernel> cudaError_t launch(const Ctx &c, uint32_t smem, const AttnArgs &a, int64_t max_tiles, int heads) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, smem, ready);
    if (e != cudaSuccess) return e;
    BwdMaps m;
    if (!bwd_maps(a, m)) return cudaErrorNotSupported;
    const int64_t items = max_tiles * heads, blocks = items < c.sms ? items : c.sms;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(THREADS), smem, c.stream, m, a, heads);
}

int take(cudaStream_t stream) {
    int v = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_dsc_status_attn_bwd, sizeof v, 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return -1;
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_dsc_status_attn_bwd, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return -1;
    return cudaStreamSynchronize(stream) == cudaSuccess ? v : -1;
}

}  // namespace
}  // namespace attn_tc

cudaError_t launch_attn_dkv_tc(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    using namespace attn_tc;
    const int heads = a.Hkv * a.nsplit;
    const cudaError_t e = a.d <= 64 ? launch<k_attn_dkv_tc<64>>(c, Dkv<64>::TOTAL, a, max_tiles, heads)
                                    : launch<k_attn_dkv_tc<128>>(c, Dkv<128>::TOTAL, a, max_tiles, heads);
    return e != cudaSuccess || a.nsplit == 1 ? e : launch_attn_dkv_sum(c, DSC_BF16, a);
}

cudaError_t launch_attn_dq_tc(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    using namespace attn_tc;
    return a.d <= 64 ? launch<k_attn_dq_tc<64>>(c, Dq<64>::TOTAL, a, max_tiles, a.Hq)
                     : launch<k_attn_dq_tc<128>>(c, Dq<128>::TOTAL, a, max_tiles, a.Hq);
}

int take_attn_bwd_status(cudaStream_t stream) { return attn_tc::take(stream); }

}  // namespace dsc
