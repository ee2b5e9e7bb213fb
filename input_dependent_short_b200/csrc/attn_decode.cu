// Attention of one new token per sequence over a paged key-value cache.
//
// A key and value is read once for a chunk of its group's query heads (16 in bf16,
// 4 in fp32; larger groups read the cache once a chunk); the time is that of
// reading them.  The lengths live on the device and may differ
// a lot, so the work is dealt out there: the cache is cut into units of 64
// tokens of one (sequence, key head, chunk of its query heads) -- a segment's
// units are consecutive -- and block c of G takes units [c U / G, (c+1) U / G).
// A block that covers a whole segment writes its result; one that covers a
// part leaves (maximum, sum, unnormalised output) in the workspace, and a
// second kernel joins each shared segment's parts in the order of their
// blocks.  A share has at most one segment that began in an earlier block
// (part 0) and one that goes on in the next (part 1).
#include "attn.cuh"

namespace dsc {
namespace {

constexpr int UNIT = 64;     // tokens of a unit
constexpr int NTH = 128;     // threads of a block
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;
// The running maximum of a token that counts is at least this, so that it tells
// "nothing to read" (-infinity: zeros) from scores that are all -infinity (a
// weights' sum of 0, and 0 / 0 as in the formula).
constexpr float LOWEST = -3.402823466e38f;

__device__ __forceinline__ int seq_len(const DecodeArgs &a, int b) {
    const int64_t n = a.seq_lens[b], most = a.max_pages * a.page;
    return (int)(n < 0 ? 0 : (n < most ? n : most));
}
__device__ __forceinline__ int seq_units(const DecodeArgs &a, int b) { return (seq_len(a, b) + UNIT - 1) / UNIT; }

// This block's share and the sequence its first unit lies in.
struct Share {
    long long u0, u1, U;  // units; U: all of them
    long long base;       // first unit of sequence b
    int G;                // blocks with work
    int b;
};

// All threads of the block; HX segments per sequence.
__device__ Share find_share(const DecodeArgs &a, int HX) {
    __shared__ long long wsum[NTH / 32];
    __shared__ Share share;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + NTH - 1) / NTH;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    long long own = 0;
    for (int b = b0; b < b1; ++b) own += seq_units(a, b);
    long long v = own;
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(FULL_MASK, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    long long before = v - own, total = 0;
    for (int w = 0; w < NTH / 32; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    const long long U = total * HX;
    const int G = (int)(U < (long long)gridDim.x ? U : (long long)gridDim.x);
    const int c = blockIdx.x;
    if (tid == 0) share = Share{0, 0, U, 0, G, 0};
    __syncthreads();
    if (c < G) {
        const long long u0 = c * U / G, u1 = (c + 1) * U / G;
        long long base = before * HX;
        if (u0 >= base && u0 < base + own * HX) {  // one thread's range holds u0
            int b = b0;
            for (;; ++b) {
                const long long n = (long long)seq_units(a, b) * HX;
                if (u0 < base + n) break;
                base += n;
            }
            share = Share{u0, u1, U, base, G, b};
        }
    }
    __syncthreads();
    return share;
}

// Zeros for the sequences with nothing to read.
template <typename T> __device__ void zero_empty(const DecodeArgs &a) {
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (seq_len(a, b)) continue;
        for (int i = threadIdx.x; i < a.Hq * a.d; i += NTH) static_cast<T *>(a.o)[(int64_t)b * a.Hq * a.d + i] = from_f<T>(0.f);
        if (a.lse)
            for (int h = threadIdx.x; h < a.Hq; h += NTH) a.lse[(int64_t)b * a.Hq + h] = -INFINITY;
    }
}

// One segment's walk: where a unit lies.
struct Place {
    long long u, base;  // the unit; the first unit of sequence b
    int b, hx, j;       // sequence, segment of it, unit of the segment
    int len, nu;        // the sequence's tokens and units
};

__device__ __forceinline__ Place place_of(const DecodeArgs &a, const Share &w, int HX) {
    Place p{w.u0, w.base, w.b, 0, 0, 0, 1};
    if (w.u0 < w.u1) {
        p.len = seq_len(a, p.b);
        p.nu = (p.len + UNIT - 1) / UNIT;
        p.hx = (int)((p.u - p.base) / p.nu);
        p.j = (int)((p.u - p.base) % p.nu);
    }
    return p;
}

__device__ __forceinline__ void next_unit(const DecodeArgs &a, Place &p, int HX) {
    ++p.u;
    if (++p.j < p.nu) return;
    p.j = 0;
    if (++p.hx < HX) return;
    p.hx = 0;
    p.base += (long long)p.nu * HX;
    do {
        if (++p.b >= a.B) return;
        p.len = seq_len(a, p.b);
    } while (!p.len);
    p.nu = (p.len + UNIT - 1) / UNIT;
}

// The warps' states of MG heads, joined.
constexpr int MG = 4;
struct Merge {
    float m[NTH / 32][MG], l[NTH / 32][MG], o[NTH / 32][MG][128];
};

// Heads h0 + g0 .. + nh-1 of a chunk: the result when this block had the whole
// segment, else its part.  All threads, between two barriers.
template <typename T>
__device__ __forceinline__ void finish_heads(const DecodeArgs &a, const Merge &s, int b, int h0, int g0, int nh, int GC,
                                             bool whole, int slot) {
    const int tid = threadIdx.x;
    for (int g = 0; g < nh; ++g) {
        float mn = -INFINITY;
        for (int k = 0; k < NTH / 32; ++k) mn = fmaxf(mn, s.m[k][g]);
        const float mu = mn == -INFINITY ? 0.f : mn;
        float ls = 0.f, os = 0.f;
        for (int k = 0; k < NTH / 32; ++k) {
            const float f = exp2f(s.m[k][g] - mu);
            ls += s.l[k][g] * f;
            if (tid < a.d) os += s.o[k][g][tid] * f;
        }
        if (whole) {
            const int64_t r = (int64_t)b * a.Hq + h0 + g0 + g;
            if (tid < a.d) static_cast<T *>(a.o)[r * a.d + tid] = from_f<T>(mn == -INFINITY ? 0.f : os / ls);
            if (tid == 0 && a.lse) a.lse[r] = mn == -INFINITY ? -INFINITY : (mn + log2f(ls)) * LN2;
        } else {
            float *p = a.part + ((int64_t)(blockIdx.x * 2 + slot) * GC + g0 + g) * (a.d + 2);
            if (tid < a.d) p[2 + tid] = os;
            if (tid == 0) {
                p[0] = mn;
                p[1] = ls;
            }
        }
    }
}

// The record of a segment that begins in this block and goes on.
__device__ __forceinline__ int4 tail_record(const Share &w, const Place &p, int h0, int nh) {
    const long long e = p.base + (long long)(p.hx + 1) * p.nu;  // the segment's end
    const int last = (int)((e * w.G - 1) / w.U);                // the block that holds unit e - 1
    return make_int4(p.b, h0, nh, last - (int)blockIdx.x + 1);
}

// ---------------------------------------------------------- CUDA cores ---
// fp32: a warp takes keys in turn: LPK lanes hold a row's 16-byte vectors, 32 / LPK
// rows at a time, STEPS of them in flight.  GC query heads share the loads.
constexpr int STEPS = 4;

template <int GC> __global__ void __launch_bounds__(NTH) k_decode_simt(DecodeArgs a, int nch, int LPK) {
    constexpr int V = VecOf<float>::V;
    __shared__ Merge mg;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPK, pos = lane % LPK, KPW = 32 / LPK;
    const bool on = pos * V < a.d;
    pdl_wait();
    pdl_trigger();
    const int HX = a.Hkv * nch;
    zero_empty<float>(a);
    const Share w = find_share(a, HX);
    int4 rec = make_int4(0, 0, 0, 0);
    Place p = place_of(a, w, HX);
    while (p.u < w.u1) {
        const int j1 = (int)min((long long)p.nu, p.j + (w.u1 - p.u));
        const int hk = p.hx / nch, h0 = hk * a.group + (p.hx % nch) * GC, nh = min(GC, hk * a.group + a.group - h0);
        float q[GC][V], o[GC][V], m[GC], l[GC];
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) q[g][e] = o[g][e] = 0.f;
            if (g < nh && on) unpack(ld16(static_cast<const float *>(a.q) + p.b * a.qs + (int64_t)(h0 + g) * a.d + pos * V), q[g]);
#pragma unroll
            for (int e = 0; e < V; ++e) q[g][e] *= a.scale * LOG2E;
        }
        const int32_t *tab = a.table + (int64_t)p.b * a.max_pages;
        const int end = min(p.len, j1 * UNIT);
        for (int t0 = p.j * UNIT + warp * KPW; t0 < end; t0 += (NTH / 32) * KPW * STEPS) {
            uint4 kv[STEPS], vv[STEPS];
            bool ok[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int t = t0 + i * (NTH / 32) * KPW + sub;
                ok[i] = false;
                kv[i] = vv[i] = make_uint4(0, 0, 0, 0);
                if (t < end) {
                    const int pg = t / a.page, page = tab[pg];
                    if (page >= 0 && page < a.n_pages) {
                        ok[i] = true;
                        const int64_t at = (((int64_t)page * a.Hkv + hk) * a.page + (t - pg * a.page)) * a.d + pos * V;
                        if (on) {
                            kv[i] = ld16(static_cast<const float *>(a.k) + at);
                            vv[i] = ld16(static_cast<const float *>(a.v) + at);
                        }
                    }
                }
            }
            float s[STEPS][GC];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                float f[V];
                unpack(kv[i], f);
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) x = fmaf(q[g][e], f[e], x);
                    s[i][g] = x;
                }
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int g = 0; g < GC; ++g) {
                    for (int k = LPK >> 1; k > 0; k >>= 1) s[i][g] += __shfl_xor_sync(FULL_MASK, s[i][g], k);
                    if (!ok[i]) s[i][g] = -INFINITY;
                }
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                float mn = m[g];
#pragma unroll
                for (int i = 0; i < STEPS; ++i) mn = fmaxf(mn, ok[i] ? fmaxf(s[i][g], LOWEST) : -INFINITY);
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[g] - mu);
                m[g] = mn;
                l[g] *= f;
#pragma unroll
                for (int e = 0; e < V; ++e) o[g][e] *= f;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    s[i][g] = exp2f(s[i][g] - mu);
                    l[g] += s[i][g];
                }
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                float f[V];
                unpack(vv[i], f);  // zeros where masked
#pragma unroll
                for (int g = 0; g < GC; ++g)
#pragma unroll
                    for (int e = 0; e < V; ++e) o[g][e] = fmaf(s[i][g], f[e], o[g][e]);
            }
        }
        // join the warp's row groups, then the warps
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            for (int k = LPK; k < 32; k <<= 1) {
                const float mo = __shfl_xor_sync(FULL_MASK, m[g], k), lo = __shfl_xor_sync(FULL_MASK, l[g], k);
                const float mn = fmaxf(m[g], mo), mu = mn == -INFINITY ? 0.f : mn;
                const float fa = exp2f(m[g] - mu), fb = exp2f(mo - mu);
                m[g] = mn;
                l[g] = l[g] * fa + lo * fb;
#pragma unroll
                for (int e = 0; e < V; ++e) o[g][e] = o[g][e] * fa + __shfl_xor_sync(FULL_MASK, o[g][e], k) * fb;
            }
        }
        __syncthreads();  // the buffer's last readers are done
        if (sub == 0) {
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                if (pos == 0) {
                    mg.m[warp][g] = m[g];
                    mg.l[warp][g] = l[g];
                }
                if (on)
#pragma unroll
                    for (int e = 0; e < V; ++e) mg.o[warp][g][pos * V + e] = o[g][e];
            }
        }
        __syncthreads();
        const bool whole = p.j == 0 && j1 == p.nu;
        finish_heads<float>(a, mg, p.b, h0, 0, nh, GC, whole, p.j == 0);
        if (p.j == 0 && !whole) rec = tail_record(w, p, h0, nh);
        p.u += j1 - p.j - 1;
        p.j = j1 - 1;
        next_unit(a, p, HX);
    }
    if (tid == 0) a.rec[blockIdx.x] = rec;
}

// -------------------------------------------------------- tensor cores ---
// bf16: the group's query heads (up to 16) are the rows of mma.sync's 16 x 8 x
// 16 products.  A warp works alone on 16 of a unit's 64 tokens: it copies their
// K and V rows into its own ring of shared memory (cp.async, rows that are
// masked or missing as zeros), two units ahead, and forms S = q K^T, the
// running softmax and O += P V from there, so nothing but the segment's end
// needs the other warps, and the copies run on across segments.
//
// Bound by memory: a unit's products take a tenth of the time its 32 KB take
// to arrive, which is why 16 rows for a group of 4 are no loss, and why
// tcgen05's 128 rows would be.
constexpr int GCM = 16;      // query heads of a chunk
constexpr int STAGES = 3;

template <int DP> struct Ring {
    static constexpr int ROW = DP * 2;                   // bytes
    static constexpr int HALF = 16 * ROW;                // 16 keys (or values)
    static constexpr int WARP = STAGES * 2 * HALF;
    static constexpr int BYTES = (NTH / 32) * WARP;
    // 16-byte chunk c of row r: chunks permuted inside 128 bytes, so that 8 rows' equal chunks lie in different banks
    __device__ static uint32_t at(int r, int c) { return (uint32_t)(r * ROW + ((c ^ (r & 7)) << 4)); }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DP> __global__ void __launch_bounds__(NTH) k_decode_mma(DecodeArgs a, int nch) {
    using R = Ring<DP>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Merge mg;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)warp * R::WARP;
    pdl_wait();
    pdl_trigger();
    const int HX = a.Hkv * nch;
    zero_empty<bf16>(a);
    const Share w = find_share(a, HX);
    int4 rec = make_int4(0, 0, 0, 0);

    // Copying runs ahead: `next` is the unit whose rows are looked up next;
    // lane r < 16 holds the element offset of row r of the unit to copy (-1: none).
    Place next = place_of(a, w, HX);
    int64_t row = -1;
    auto look_up = [&]() {
        row = -1;
        if (next.u >= w.u1) return;
        const int t = next.j * UNIT + warp * 16 + (lane & 15);
        if (t < next.len) {
            const int pg = t / a.page, page = a.table[(int64_t)next.b * a.max_pages + pg];
            if (page >= 0 && page < a.n_pages)
                row = (((int64_t)page * a.Hkv + next.hx / nch) * a.page + (t - pg * a.page)) * a.d;
        }
        next_unit(a, next, HX);
    };
    u64 seen = 0;  // 16 bits a stage: its rows that count
    auto copy = [&](int s) {  // the looked-up unit into stage s; one group, empty or not
        constexpr int NV = DP / 8, RPI = 32 / NV;  // 16-byte vectors of a row, rows per instruction
        const int c = lane % NV;
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += RPI) {
            const int r = r0 + lane / NV;
            const int64_t off = __shfl_sync(FULL_MASK, row, r);
            const bool on = off >= 0 && c * 8 < a.d;
            const int64_t src = on ? off + c * 8 : 0;
            const uint32_t dst = ring + (uint32_t)(s * 2 * R::HALF) + R::at(r, c);
            cp16(dst, static_cast<const bf16 *>(a.k) + src, on);
            cp16(dst + R::HALF, static_cast<const bf16 *>(a.v) + src, on);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const u64 mask = __ballot_sync(FULL_MASK, row >= 0) & 0xffffu;
        seen = (seen & ~((u64)0xffff << (16 * s))) | mask << (16 * s);
    };
    look_up();
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        copy(s);
        look_up();
    }

    Place p = place_of(a, w, HX);
    const float c2 = a.scale * LOG2E;
    uint32_t q[DP / 16][4];
    float o[DP / 8][4], m[2], l[2];
    int stage = 0, h0 = 0, nh = 0, jfirst = 0;
    bool fresh = true;
    while (p.u < w.u1) {
        if (fresh) {  // a new segment: its queries, an empty state
            fresh = false;
            jfirst = p.j;
            const int hk = p.hx / nch;
            h0 = hk * a.group + (p.hx % nch) * GCM;
            nh = min(GCM, hk * a.group + a.group - h0);
            const bf16 *qp = static_cast<const bf16 *>(a.q) + p.b * a.qs + (int64_t)h0 * a.d;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = (lane >> 2) + 8 * (e & 1), c = 16 * k + 2 * (lane & 3) + 8 * (e >> 1);
                    q[k][e] = r < nh && c < a.d ? *reinterpret_cast<const uint32_t *>(qp + r * a.d + c) : 0u;
                }
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
        }
        // the stage read in the last turn takes the unit two ahead
        copy(stage == 0 ? STAGES - 1 : stage - 1);
        const uint32_t mask = (uint32_t)(seen >> (16 * stage)) & 0xffffu;
        look_up();
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();
        const uint32_t kb = ring + (uint32_t)(stage * 2 * R::HALF), vb = kb + R::HALF;
        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            // matrices: keys 0-7 and 8-15, elements 16 k + 0-7 and 8-15
            uint32_t b[4];
            ldsm4(b, kb + R::at((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
            mma16816(s[0], q[k], b[0], b[1]);
            mma16816(s[1], q[k], b[2], b[3]);
        }
        // rows lane / 4 (e = 0, 1) and + 8 (e = 2, 3); tokens 8 n + 2 (lane % 4) + (e & 1)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[n][e] = (mask >> (8 * n + 2 * (lane & 3) + (e & 1))) & 1u ? s[n][e] * c2 : -INFINITY;
        float f[2];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float t = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            t = fmaxf(t, __shfl_xor_sync(FULL_MASK, t, 1));
            t = fmaxf(t, __shfl_xor_sync(FULL_MASK, t, 2));
            const float mn = fmaxf(fmaxf(m[r], t), mask ? LOWEST : -INFINITY);
            f[r] = m[r] == mn ? 1.f : exp2f(m[r] - mn);
            moved |= m[r] != mn;
            m[r] = mn;
            const float mu = mn == -INFINITY ? 0.f : mn;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[n][2 * r + e] = exp2f(s[n][2 * r + e] - mu);
                    sum += s[n][2 * r + e];
                }
            l[r] = l[r] * f[r] + sum;  // this lane's tokens; joined at the end
        }
        if (__any_sync(FULL_MASK, moved)) {
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                o[n][0] *= f[0];
                o[n][1] *= f[0];
                o[n][2] *= f[1];
                o[n][3] *= f[1];
            }
        }
        const uint32_t pa[4] = {pack_bf2(s[0][0], s[0][1]), pack_bf2(s[0][2], s[0][3]), pack_bf2(s[1][0], s[1][1]),
                                pack_bf2(s[1][2], s[1][3])};
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
            // matrices: tokens 0-7 and 8-15 of elements 16 n + 0-7, then of 8-15
            uint32_t b[4];
            ldsm4t(b, vb + R::at((lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
            mma16816(o[2 * n], pa, b[0], b[1]);
            mma16816(o[2 * n + 1], pa, b[2], b[3]);
        }
        __syncwarp();  // the stage is read before it is filled again
        stage = stage + 1 == STAGES ? 0 : stage + 1;

        if (p.j + 1 == p.nu || p.u + 1 == w.u1) {  // the segment ends here, or this block's part of it
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(FULL_MASK, l[r], 1);
                l[r] += __shfl_xor_sync(FULL_MASK, l[r], 2);
            }
            const bool whole = jfirst == 0 && p.j + 1 == p.nu;
            for (int g0 = 0; g0 < nh; g0 += MG) {
                __syncthreads();
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int g = (lane >> 2) + 8 * r - g0;
                    if (g < 0 || g >= MG) continue;
                    if ((lane & 3) == 0) {
                        mg.m[warp][g] = m[r];
                        mg.l[warp][g] = l[r];
                    }
#pragma unroll
                    for (int n = 0; n < DP / 8; ++n)
                        *reinterpret_cast<float2 *>(&mg.o[warp][g][8 * n + 2 * (lane & 3)]) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
                }
                __syncthreads();
                finish_heads<bf16>(a, mg, p.b, h0, g0, min(MG, nh - g0), GCM, whole, jfirst == 0);
            }
            if (jfirst == 0 && !whole) rec = tail_record(w, p, h0, nh);
            fresh = true;
        }
        next_unit(a, p, HX);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 0) a.rec[blockIdx.x] = rec;
}

// Joins the parts of the segment that begins in block c's share and goes on:
// part 1 of block c, part 0 of the next rec.w - 1 blocks.  blockIdx.y: head.
// JG groups of 128 threads (a thread a column) take every JG-th part, and their
// sums are added in the groups' order.
constexpr int JG = 4;

template <typename T, int GC> __global__ void __launch_bounds__(128 * JG) k_decode_join(DecodeArgs a) {
    __shared__ float red[4 * JG], sl[JG], so[JG][128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = tid & 127, grp = tid >> 7;
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, g = blockIdx.y;
    const int4 rec = a.rec[c];
    if (g >= rec.z) return;
    const int n = rec.w;
    const int64_t pitch = (int64_t)GC * (a.d + 2);
    // part i of the segment
    auto part = [&](int i) { return a.part + ((int64_t)(c + i) * 2 + (i == 0)) * pitch + (int64_t)g * (a.d + 2); };
    float mn = -INFINITY;
    for (int i = tid; i < n; i += 128 * JG) mn = fmaxf(mn, part(i)[0]);
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(FULL_MASK, mn, o));
    if (lane == 0) red[warp] = mn;
    __syncthreads();
    for (int k = 0; k < 4 * JG; ++k) mn = fmaxf(mn, red[k]);
    const float mu = mn == -INFINITY ? 0.f : mn;
    float ls = 0.f, os = 0.f;
#pragma unroll 4
    for (int i = grp; i < n; i += JG) {
        const float *p = part(i);
        const float f = exp2f(p[0] - mu);
        ls += p[1] * f;
        if (col < a.d) os += p[2 + col] * f;
    }
    if (col == 0) sl[grp] = ls;
    so[grp][col] = os;
    __syncthreads();
    if (grp) return;
    ls = os = 0.f;
#pragma unroll
    for (int k = 0; k < JG; ++k) {
        ls += sl[k];
        os += so[k][col];
    }
    const int64_t r = (int64_t)rec.x * a.Hq + rec.y + g;
    if (col < a.d) static_cast<T *>(a.o)[r * a.d + col] = from_f<T>(mn == -INFINITY ? 0.f : os / ls);
    if (col == 0 && a.lse) a.lse[r] = mn == -INFINITY ? -INFINITY : (mn + log2f(ls)) * LN2;
}

// Four blocks per SM; two where the rings of 128 elements fill the shared memory.
int grid_blocks(const Ctx &c, int dtype, int d) { return c.sms * (dtype == DSC_BF16 && d > 64 ? 2 : 4); }

template <typename T, int GC> cudaError_t launch_join(const Ctx &c, const DecodeArgs &a, int blocks) {
    return launch_pdl(k_decode_join<T, GC>, dim3((unsigned)blocks, (unsigned)(a.group < GC ? a.group : GC)), dim3(128 * JG), 0,
                      c.stream, a);
}

template <int GC> cudaError_t launch_simt(const Ctx &c, const DecodeArgs &a) {
    constexpr int V = VecOf<float>::V;
    int LPK = 1;
    while (LPK < 32 && LPK * V < a.d) LPK <<= 1;
    const int nch = (a.group + GC - 1) / GC, blocks = grid_blocks(c, DSC_F32, a.d);
    const cudaError_t e = launch_pdl(k_decode_simt<GC>, dim3((unsigned)blocks), dim3(NTH), 0, c.stream, a, nch, LPK);
    return e != cudaSuccess ? e : launch_join<float, GC>(c, a, blocks);
}

template <int DP> cudaError_t launch_mma(const Ctx &c, const DecodeArgs &a) {
    const int nch = (a.group + GCM - 1) / GCM, blocks = grid_blocks(c, DSC_BF16, a.d);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem(k_decode_mma<DP>, Ring<DP>::BYTES, ready);
    if (e == cudaSuccess) e = launch_pdl(k_decode_mma<DP>, dim3((unsigned)blocks), dim3(NTH), Ring<DP>::BYTES, c.stream, a, nch);
    return e != cudaSuccess ? e : launch_join<bf16, GCM>(c, a, blocks);
}

size_t rec_bytes(const Ctx &c, int dtype, int d) { return ((size_t)grid_blocks(c, dtype, d) * sizeof(int4) + 255) & ~(size_t)255; }

}  // namespace

size_t decode_attn_ws_bytes(const Ctx &c, int dtype, int d) {
    const size_t gc = dtype == DSC_BF16 ? GCM : MG;
    return rec_bytes(c, dtype, d) + (size_t)grid_blocks(c, dtype, d) * 2 * gc * (size_t)(d + 2) * sizeof(float);
}

cudaError_t launch_decode_attn(const Ctx &c, int dtype, DecodeArgs a, void *ws) {
    a.rec = static_cast<int4 *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + rec_bytes(c, dtype, a.d));
    if (dtype == DSC_BF16) return a.d <= 64 ? launch_mma<64>(c, a) : launch_mma<128>(c, a);
    if (a.group == 1) return launch_simt<1>(c, a);
    if (a.group == 2) return launch_simt<2>(c, a);
    return launch_simt<4>(c, a);
}

}  // namespace dsc
