// Attention over packed documents on the CUDA cores: the fp32 path.
//
// One block of 128 threads takes 32 rows of one document and one head (query
// rows, or keys for dk and dv) and walks the other side in tiles of 64, all
// operands in shared memory.  Thread (ty, tx) of an 8 x 16 grid owns rows
// 4 ty + 0..3 and columns tx + 16 j of a 32 x 64 score tile, and elements
// 4 tx + 64 c + 0..3 of its rows' outputs.  The softmax is one pass with a
// running maximum and sum; rows are joined over the 16 tx lanes by shuffles.
//
// 32 rows rather than 64 (with 256 threads): a training step of 1500 tokens and
// 8 heads of 64 has too few tiles of 64 to fill the GPU and three to four
// blocks of this size share an SM, so one's loads run under another's products.
// Bound by the loads from shared memory (a 4 x 4 thread tile reads 32 fp32 for 64
// products: that pipe is 76 to 84 % busy, the FMA pipe 55 to 58 %): 4096 tokens,
// 8 heads of 64, forward 524 us and gradients 1626 us (33 and 26 of 72 TFLOP/s).
//
// Operand rows outside the document are zeros, never what memory holds there,
// and a masked probability is an exact zero that is not multiplied with
// anything: on the diagonal tile each thread leaves the masked keys out, so a
// NaN or infinity behind a row does not reach it.
#include "attn.cuh"

namespace dsc {
namespace {

constexpr int BM = SIMT_ROWS;   // rows of the block's own tile
constexpr int BN = 64;          // rows of the tiles it walks
constexpr int NTHR = 128;
constexpr int PP = BN + 4;      // pitch of a probability tile (floats)
constexpr float LOG2E = 1.4426950408889634f;

template <int DP> struct Smem {
    static constexpr int PITCH = DP + 4;  // an operand row: 16-byte aligned, rows 4 banks apart
    static constexpr int OWN = BM * PITCH, WALK = BN * PITCH, PROB = BM * PP;
};

// R rows of one head into shared memory: zero for rows >= n and columns >= d.
template <int DP, int R> __device__ __forceinline__ void load_tile(float *s, const float *g, int64_t stride, int n, int d, int tid) {
    constexpr int PITCH = Smem<DP>::PITCH;
#pragma unroll 8
    for (int i = tid; i < R * (DP / 4); i += NTHR) {
        const int r = i / (DP / 4), c = (i % (DP / 4)) * 4;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < n && c < d) x = ld16(g + r * stride + c);
        *reinterpret_cast<uint4 *>(s + r * PITCH + c) = x;
    }
}

// 16 bytes of shared memory as two fp32 pairs.
struct Pair2 {
    u64 a, b;
};
__device__ __forceinline__ Pair2 ld_pairs(const float *p) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(p);
    return Pair2{x.x, x.y};
}

// acc[i][j] = sum_c A[4 ty + i][c] * B[tx + 16 j][c], the even and the odd c
// apart (fma.rn.f32x2: half the instructions, which leaves issue slots for the
// loads).
template <int DP>
__device__ __forceinline__ void tile_dot(float (&acc)[4][4], const float *A, const float *B, int ty, int tx) {
    constexpr int PITCH = Smem<DP>::PITCH;
    u64 sum[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = 0;
#pragma unroll 4
    for (int c = 0; c < DP; c += 4) {
        Pair2 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = ld_pairs(A + (4 * ty + i) * PITCH + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = ld_pairs(B + (tx + 16 * j) * PITCH + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i][j] = fma2(a[i].b, b[j].b, fma2(a[i].a, b[j].a, sum[i][j]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = lo2(sum[i][j]) + hi2(sum[i][j]);
}

// out[i][2 c + e], pairs: elements 4 tx + 64 c + 2 e and + 1 of row 4 ty + i, +=
// sum_k P[4 ty + i][k] * B[k][...].  DIAG: only the k of the row, k <= 4 ty + i + off,
// or k >= 4 ty + i when `upper`.
template <int DP, bool DIAG>
__device__ __forceinline__ void tile_acc(u64 (&out)[4][DP / 32], const float *P, const float *B, int ty, int tx,
                                         bool upper, int off) {
    constexpr int PITCH = Smem<DP>::PITCH, NC = DP / 64;
#pragma unroll 2
    for (int k = 0; k < BN; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(P + (4 * ty + i) * PP + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            Pair2 b[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) b[c] = ld_pairs(B + (k + e) * PITCH + 4 * tx + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = e == 0 ? p[i].x : (e == 1 ? p[i].y : (e == 2 ? p[i].z : p[i].w));
                if (DIAG && (upper ? k + e < 4 * ty + i : k + e > 4 * ty + i + off)) continue;
                const u64 w = mk2(x, x);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    out[i][2 * c] = fma2(w, b[c].a, out[i][2 * c]);
                    out[i][2 * c + 1] = fma2(w, b[c].b, out[i][2 * c + 1]);
                }
            }
        }
    }
}

// The block's tile and head: tiles in the list's order, all heads of one before
// the next, so the dearest items of every head start first.  Tile after tile of
// one head before the next head was slower (4096 tokens, 8 heads of 64: gradients
// 2150 us against 1626; 700 tokens: 204 against 174), but for the gradients
// at sizes whose blocks all fit at once (1500 tokens: 500 against 520).
__device__ __forceinline__ bool take_item(const AttnArgs &a, int heads, AttnTile &t, int &h) {
    const int i = blockIdx.x / heads;
    if (i >= *a.list.count) return false;
    t = a.list.tiles[i];
    h = blockIdx.x % heads;
    return true;
}

// Rows r < n of the block's tile from the accumulators, times f[i].
template <int DP>
__device__ __forceinline__ void store_tile(float *g, int64_t stride, const u64 (&out)[4][DP / 32], const float (&f)[4],
                                           int n, int d, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= n) continue;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
            const int col = 4 * tx + 64 * c;
            if (col >= d) continue;
            const u64 v[2] = {mul2(out[i][2 * c], mk2(f[i], f[i])), mul2(out[i][2 * c + 1], mk2(f[i], f[i]))};
            st16(g + r * stride + col, Pairs<float>::pack(v));
        }
    }
}

__device__ __forceinline__ void zero_rows(float *g, int64_t stride, int n, int d, int tid) {
    for (int i = tid; i < n * (d / 4); i += NTHR) st16(g + (i / (d / 4)) * stride + (i % (d / 4)) * 4, make_uint4(0, 0, 0, 0));
}

// max and sum over the 16 lanes that share a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}

template <int DP> __global__ void __launch_bounds__(NTHR) k_attn_fwd_simt(AttnArgs a) {
    extern __shared__ __align__(16) float smem[];
    float *Q = smem, *K = Q + Smem<DP>::OWN, *V = K + Smem<DP>::WALK, *P = V + Smem<DP>::WALK;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_wait();
    pdl_trigger();
    AttnTile t;
    int h;
    if (!take_item(a, a.Hq, t, h)) return;
    const int hk = h / a.group;
    float *o = static_cast<float *>(a.o);
    const int64_t os = (int64_t)a.Hq * a.d;
    if (t.len < 0) {
        zero_rows(o + t.start * os + (int64_t)h * a.d, os, -t.len, a.d, tid);
        for (int r = tid; r < -t.len; r += NTHR) a.lse[h * a.T + t.start + r] = -INFINITY;
        return;
    }
    const int64_t row0 = (int64_t)t.start + t.r0;
    const int n = min(BM, t.len - t.r0);
    const float *q = static_cast<const float *>(a.q) + row0 * a.qs + (int64_t)h * a.d;
    const float *k = static_cast<const float *>(a.k) + (int64_t)t.start * a.ks + (int64_t)hk * a.d;
    const float *v = static_cast<const float *>(a.v) + (int64_t)t.start * a.vs + (int64_t)hk * a.d;
    load_tile<DP, BM>(Q, q, a.qs, n, a.d, tid);
    float m[4], l[4], one[4];
    u64 acc[4][DP / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) acc[i][c] = 0;
    }
    const float c2 = a.scale * LOG2E;
    const int top = t.r0 / BN * BN, off = t.r0 - top;  // the diagonal tile, first: every row sees a key in it
    for (int k0 = top; k0 >= 0; k0 -= BN) {
        __syncthreads();
        load_tile<DP, BN>(K, k + k0 * a.ks, a.ks, min(BN, t.len - k0), a.d, tid);
        load_tile<DP, BN>(V, v + k0 * a.vs, a.vs, min(BN, t.len - k0), a.d, tid);
        __syncthreads();
        const bool diag = k0 == top;
        float s[4][4];
        tile_dot<DP>(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mt = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (diag && tx + 16 * j > 4 * ty + i + off) s[i][j] = -INFINITY;
                mt = fmaxf(mt, s[i][j]);
            }
            const float mn = fmaxf(m[i], row_max(mt));
            const float mu = mn == -INFINITY ? 0.f : mn;  // no finite score so far
            const float f = exp2f((m[i] - mu) * c2);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f((s[i][j] - mu) * c2);
                sum += p;
                P[(4 * ty + i) * PP + tx + 16 * j] = p;
            }
            l[i] = l[i] * f + sum;  // this lane's columns; joined at the end
            m[i] = mn;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) acc[i][c] = mul2(acc[i][c], mk2(f, f));
        }
        __syncwarp();  // a row's probabilities are written and read by the same half warp
        if (diag) tile_acc<DP, true>(acc, P, V, ty, tx, false, off);
        else tile_acc<DP, false>(acc, P, V, ty, tx, false, off);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sum = row_sum(l[i]);
        one[i] = 1.f / sum;
        if (tx == 0 && 4 * ty + i < n) a.lse[h * a.T + row0 + 4 * ty + i] = m[i] * a.scale + logf(sum);
    }
    store_tile<DP>(o + row0 * os + (int64_t)h * a.d, os, acc, one, n, a.d, ty, tx);
}

// dS = P (dP - D) of a query row and key; a masked pair gives zeros.
__device__ __forceinline__ void pair_grads(float &s, float &g, bool seen, float lse2, float delta, float c2) {
    const float p = seen ? exp2f(s * c2 - lse2) : 0.f;
    g = seen ? p * (g - delta) : 0.f;
    s = p;
}

template <int DP> __global__ void __launch_bounds__(NTHR) k_attn_dq_simt(AttnArgs a) {
    extern __shared__ __align__(16) float smem[];
    float *Q = smem, *G = Q + Smem<DP>::OWN, *K = G + Smem<DP>::OWN, *V = K + Smem<DP>::WALK, *P = V + Smem<DP>::WALK;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_wait();
    pdl_trigger();
    AttnTile t;
    int h;
    if (!take_item(a, a.Hq, t, h)) return;
    const int hk = h / a.group;
    float *dq = static_cast<float *>(a.dq) + (int64_t)h * a.d;
    if (t.len < 0) {
        zero_rows(dq + t.start * a.dqs, a.dqs, -t.len, a.d, tid);
        return;
    }
    const int64_t row0 = (int64_t)t.start + t.r0, os = (int64_t)a.Hq * a.d;
    const int n = min(BM, t.len - t.r0);
    const float *k = static_cast<const float *>(a.k) + (int64_t)t.start * a.ks + (int64_t)hk * a.d;
    const float *v = static_cast<const float *>(a.v) + (int64_t)t.start * a.vs + (int64_t)hk * a.d;
    load_tile<DP, BM>(Q, static_cast<const float *>(a.q) + row0 * a.qs + (int64_t)h * a.d, a.qs, n, a.d, tid);
    load_tile<DP, BM>(G, static_cast<const float *>(a.dout) + row0 * os + (int64_t)h * a.d, os, n, a.d, tid);
    float lse2[4], delta[4], f[4];
    u64 acc[4][DP / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;  // a row behind the document: lse = +inf makes its probabilities zero
        lse2[i] = r < n ? a.lse[h * a.T + row0 + r] * LOG2E : INFINITY;
        delta[i] = r < n ? a.delta[h * a.T + row0 + r] : 0.f;
        f[i] = a.scale;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) acc[i][c] = 0;
    }
    const int top = t.r0 / BN * BN, off = t.r0 - top;
    for (int k0 = top; k0 >= 0; k0 -= BN) {
        __syncthreads();
        load_tile<DP, BN>(K, k + k0 * a.ks, a.ks, min(BN, t.len - k0), a.d, tid);
        load_tile<DP, BN>(V, v + k0 * a.vs, a.vs, min(BN, t.len - k0), a.d, tid);
        __syncthreads();
        const bool diag = k0 == top;
        float s[4][4], g[4][4];
        tile_dot<DP>(s, Q, K, ty, tx);
        tile_dot<DP>(g, G, V, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pair_grads(s[i][j], g[i][j], !diag || tx + 16 * j <= 4 * ty + i + off, lse2[i], delta[i], a.scale * LOG2E);
                P[(4 * ty + i) * PP + tx + 16 * j] = g[i][j];
            }
        __syncwarp();
        if (diag) tile_acc<DP, true>(acc, P, K, ty, tx, false, off);
        else tile_acc<DP, false>(acc, P, K, ty, tx, false, off);
    }
    store_tile<DP>(dq + row0 * a.dqs, a.dqs, acc, f, n, a.d, ty, tx);
}

// One block owns 32 keys of one key head and adds up over (its share of) the
// group's query heads and all later query tiles, so dk and dv need no atomics.
template <int DP> __global__ void __launch_bounds__(NTHR) k_attn_dkv_simt(AttnArgs a) {
    extern __shared__ __align__(16) float smem[];
    float *K = smem, *V = K + Smem<DP>::OWN, *Q = V + Smem<DP>::OWN, *G = Q + Smem<DP>::WALK, *P = G + Smem<DP>::WALK,
          *D = P + Smem<DP>::PROB;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_wait();
    pdl_trigger();
    AttnTile t;
    int hs;
    if (!take_item(a, a.Hkv * a.nsplit, t, hs)) return;
    const int hk = hs / a.nsplit, sp = hs % a.nsplit, gs = a.group / a.nsplit;
    const bool parts = a.nsplit > 1;
    const int64_t ps = (int64_t)a.Hkv * a.d, po = ((int64_t)sp * a.T * a.Hkv + hk) * a.d;
    float *dk = parts ? a.kpart + po : static_cast<float *>(a.dk) + (int64_t)hk * a.d;
    float *dv = parts ? a.vpart + po : static_cast<float *>(a.dv) + (int64_t)hk * a.d;
    const int64_t dks = parts ? ps : a.dks, dvs = parts ? ps : a.dvs;
    if (t.len < 0) {
        zero_rows(dk + t.start * dks, dks, -t.len, a.d, tid);
        zero_rows(dv + t.start * dvs, dvs, -t.len, a.d, tid);
        return;
    }
    const int64_t row0 = (int64_t)t.start + t.r0, os = (int64_t)a.Hq * a.d;
    const int n = min(BM, t.len - t.r0);
    load_tile<DP, BM>(K, static_cast<const float *>(a.k) + row0 * a.ks + (int64_t)hk * a.d, a.ks, n, a.d, tid);
    load_tile<DP, BM>(V, static_cast<const float *>(a.v) + row0 * a.vs + (int64_t)hk * a.d, a.vs, n, a.d, tid);
    float fk[4], fv[4];
    u64 gk[4][DP / 32], gv[4][DP / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        fk[i] = parts ? 1.f : a.scale;
        fv[i] = 1.f;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) gk[i][c] = gv[i][c] = 0;
    }
    for (int hh = 0; hh < gs; ++hh) {
        const int h = hk * a.group + sp * gs + hh;
        const float *q = static_cast<const float *>(a.q) + (int64_t)t.start * a.qs + (int64_t)h * a.d;
        const float *g = static_cast<const float *>(a.dout) + (int64_t)t.start * os + (int64_t)h * a.d;
        for (int q0 = t.r0; q0 < t.len; q0 += BN) {
            const int nq = min(BN, t.len - q0);
            __syncthreads();
            load_tile<DP, BN>(Q, q + q0 * a.qs, a.qs, nq, a.d, tid);
            load_tile<DP, BN>(G, g + q0 * os, os, nq, a.d, tid);
            float lse2[4], delta[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = tx + 16 * j;
                const int64_t at = h * a.T + t.start + q0 + r;
                lse2[j] = r < nq ? a.lse[at] * LOG2E : INFINITY;
                delta[j] = r < nq ? a.delta[at] : 0.f;
            }
            __syncthreads();
            const bool diag = q0 == t.r0;
            float s[4][4], w[4][4];  // rows: keys, columns: queries
            tile_dot<DP>(s, K, Q, ty, tx);
            tile_dot<DP>(w, V, G, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    pair_grads(s[i][j], w[i][j], !diag || tx + 16 * j >= 4 * ty + i, lse2[j], delta[j], a.scale * LOG2E);
                    P[(4 * ty + i) * PP + tx + 16 * j] = s[i][j];
                    D[(4 * ty + i) * PP + tx + 16 * j] = w[i][j];
                }
            __syncwarp();
            if (diag) {
                tile_acc<DP, true>(gv, P, G, ty, tx, true, 0);
                tile_acc<DP, true>(gk, D, Q, ty, tx, true, 0);
            } else {
                tile_acc<DP, false>(gv, P, G, ty, tx, true, 0);
                tile_acc<DP, false>(gk, D, Q, ty, tx, true, 0);
            }
        }
    }
    store_tile<DP>(dk + row0 * dks, dks, gk, fk, n, a.d, ty, tx);
    store_tile<DP>(dv + row0 * dvs, dvs, gv, fv, n, a.d, ty, tx);
}

template <auto kernel> cudaError_t launch(const Ctx &c, const AttnArgs &a, int64_t max_tiles, int heads, size_t smem) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, smem, ready);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)(max_tiles * heads)), dim3(NTHR), smem, c.stream, a);
}

template <int DP> constexpr size_t smem_bytes(int own, int probs) {
    return (size_t)(own * Smem<DP>::OWN + 2 * Smem<DP>::WALK + probs * Smem<DP>::PROB) * sizeof(float);
}

}  // namespace

cudaError_t launch_attn_fwd_simt(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    return a.d <= 64 ? launch<k_attn_fwd_simt<64>>(c, a, max_tiles, a.Hq, smem_bytes<64>(1, 1))
                     : launch<k_attn_fwd_simt<128>>(c, a, max_tiles, a.Hq, smem_bytes<128>(1, 1));
}

cudaError_t launch_attn_dq_simt(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    return a.d <= 64 ? launch<k_attn_dq_simt<64>>(c, a, max_tiles, a.Hq, smem_bytes<64>(2, 1))
                     : launch<k_attn_dq_simt<128>>(c, a, max_tiles, a.Hq, smem_bytes<128>(2, 1));
}

cudaError_t launch_attn_dkv_simt(const Ctx &c, const AttnArgs &a, int64_t max_tiles) {
    const cudaError_t e = a.d <= 64 ? launch<k_attn_dkv_simt<64>>(c, a, max_tiles, a.Hkv * a.nsplit, smem_bytes<64>(2, 2))
                                    : launch<k_attn_dkv_simt<128>>(c, a, max_tiles, a.Hkv * a.nsplit, smem_bytes<128>(2, 2));
    return e != cudaSuccess || a.nsplit == 1 ? e : launch_attn_dkv_sum(c, DSC_F32, a);
}

}  // namespace dsc
