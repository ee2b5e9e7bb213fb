// The tile list of packed documents, the fp32 backward's row sums, and the sum of dk's and dv's parts.
//
// The host does not know the documents' lengths (they are offsets on the
// device), so one block turns them into a list of tiles, sorted so that the
// expensive tiles come first: with the cheap ones last the SMs finish together.
#include "attn.cuh"

namespace dsc {
namespace {

constexpr int NBIN = 1024;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Counting sort: a histogram of the tiles' keys, its running sum from the
// largest key down, then every tile takes the next place of its bin.  The places
// inside a bin depend on the order of the atomics, and only the order in which
// blocks run depends on them.  One warp per document, lanes over its tiles.
//
// The key is the tile's cost (the best balance) where the inputs fit L2.  Where
// they do not, it is the document's number of tiles, and a document's tiles take
// consecutive places, the most expensive first: they read the same keys and
// values, or queries and gradients.  (23 documents, 16 heads of 128, 268 MB:
// by cost half of the reads missed L2 and the inputs were read 1.6 times;
// gradients 336 us by cost, 302 by document.  7 documents, 20 MB, forward and
// gradients: 114 us by cost, 127 by document.)
//
// Documents that do not overlap have `cap` tiles at most.  Offsets that go back
// and forth can ask for any number (2^23 documents of 2^30 rows: 2^48 tiles):
// each warp stops counting once it is above cap, and a total above it counts as
// no documents at all, so neither the sums nor the time can run away.
__global__ void __launch_bounds__(1024) k_attn_tiles(const int32_t *__restrict__ cu, int n_docs, int T, int rows,
                                                     int shift, int by_doc, int cap, int *__restrict__ rising,
                                                     int *__restrict__ falling_list) {
    __shared__ int hist[NBIN];
    __shared__ int wsum[32];
    __shared__ long long wtiles[32];
    __shared__ bool overlap;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool falling = blockIdx.x == 1;
    int *count = falling ? falling_list : rising;
    AttnTile *tiles = reinterpret_cast<AttnTile *>(count + 4);
    hist[tid] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    int begin = clampi(cu[0], 0, T);
    int last = begin;  // end of the last document
    for (int pass = 0; pass < 2; ++pass) {
        long long mine = 0;  // this warp's tiles
        for (int s = warp; s < n_docs; s += 32) {
            const int a = clampi(cu[s], 0, T), b = clampi(cu[s + 1], a, T);
            last = max(last, b);
            const int nt = (b - a + rows - 1) / rows;
            mine += nt;
            if (mine > cap) break;
            int first = 0;
            if (by_doc) {
                if (lane == 0) first = atomicAdd(&hist[min(nt >> shift, NBIN - 1)], nt);
                first = __shfl_sync(FULL_MASK, first, 0);
            }
            for (int j = lane; j < nt; j += 32) {
                const int cost = falling ? nt - 1 - j : j;
                const int i = by_doc ? first + nt - 1 - cost : atomicAdd(&hist[min(cost >> shift, NBIN - 1)], 1);
                if (pass && i >= 0 && i < cap) tiles[i] = AttnTile{a, b - a, j * rows, 0};
            }
        }
        if (pass == 0 && lane == 0) wtiles[warp] = mine;
        __syncthreads();
        if (pass == 0) {  // hist[b] <- tiles in the bins above b
            const int bin = NBIN - 1 - tid;
            const int own = hist[bin];
            int v = own;
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(FULL_MASK, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) wsum[warp] = v;
            __syncthreads();
            if (warp == 0) {
                int w = wsum[lane];
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(FULL_MASK, w, o);
                    if (lane >= o) w += u;
                }
                wsum[lane] = w;
                long long n = wtiles[lane];
                for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(FULL_MASK, n, o);
                if (lane == 0) overlap = n > cap;
            }
            __syncthreads();
            if (overlap) break;
            hist[bin] = v - own + (warp ? wsum[warp - 1] : 0);
            __syncthreads();
        }
    }
    // rows before the first and behind the last document
    last = __reduce_max_sync(FULL_MASK, last);
    if (lane == 0) wsum[warp] = last;
    __syncthreads();
    last = __reduce_max_sync(FULL_MASK, wsum[lane]);
    if (overlap) begin = last = T;
    const int total = overlap ? 0 : hist[0];  // bin 0 is filled last, so its running place is the number of tiles
    const int nf = (begin + rows - 1) / rows, nb = (T - last + rows - 1) / rows;
    for (int i = tid; i < nf + nb; i += 1024) {
        const int s = i < nf ? i * rows : last + (i - nf) * rows, e = i < nf ? begin : T;
        if (total + i < cap) tiles[total + i] = AttnTile{s, -min(rows, e - s), 0, 0};
    }
    if (tid == 0) {
        count[0] = min(total + nf + nb, cap);
        count[1] = 0;
    }
}

// L lanes of 16 bytes cover a head; a warp takes 4 x 32 / L consecutive (row,
// head) pairs at a time, all their loads in flight before the first sum.
__global__ void __launch_bounds__(256) k_attn_delta(const float *__restrict__ o, const float *__restrict__ dout,
                                                    float *__restrict__ delta, int64_t rows, int Hq, int d, int L) {
    constexpr int V = VecOf<float>::V, U = 4;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, per = 32 / L, sub = lane / L, pos = lane % L;
    const int64_t n = rows * Hq, step = (int64_t)gridDim.x * 8 * per * U;
    for (int64_t i = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * per * U + sub; i - sub < n; i += step) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = i + u * per;
            x[u] = y[u] = make_uint4(0, 0, 0, 0);
            if (r < n && pos * V < d) {
                x[u] = ld16(o + r * d + pos * V);
                y[u] = ld16(dout + r * d + pos * V);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float a[V], b[V], s = 0.f;
            unpack(x[u], a);
            unpack(y[u], b);
#pragma unroll
            for (int e = 0; e < V; ++e) s = fmaf(a[e], b[e], s);
            for (int k = L >> 1; k > 0; k >>= 1) s += __shfl_xor_sync(FULL_MASK, s, k);
            const int64_t r = i + u * per;
            if (pos == 0 && r < n) {
                const int64_t t = r / Hq;
                delta[(r - t * Hq) * rows + t] = s;
            }
        }
    }
}

// dk = scale * sum of the parts, dv = sum of the parts, in the parts' order.
// I: an index type that holds the number of 16-byte vectors (the divisions are
// most of the work: 64-bit ones halved the bandwidth).
template <typename T, typename I> __global__ void __launch_bounds__(256) k_attn_dkv_sum(AttnArgs a) {
    pdl_wait();
    pdl_trigger();
    const I nv = (I)(a.d / 4), heads = (I)a.Hkv, rows = (I)a.T * heads, half = rows * nv;
    const int64_t pitch = a.T * a.Hkv * a.d;
    for (I i = (I)blockIdx.x * 256 + threadIdx.x; i < 2 * half; i += (I)gridDim.x * 256) {
        const bool isk = i >= half;
        const I e = isk ? i - half : i, r = e / nv, t = r / heads, c = (e - r * nv) * 4;
        const float *part = (isk ? a.kpart : a.vpart) + (int64_t)r * a.d + c;
        float s[4] = {};
#pragma unroll 4
        for (int k = 0; k < a.nsplit; ++k) {
            float x[4];
            unpack(ld16(part + k * pitch), x);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += x[j];
        }
        const float f = isk ? a.scale : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] *= f;
        store_row<T, 4>(static_cast<T *>(isk ? a.dk : a.dv) + (int64_t)t * (isk ? a.dks : a.dvs) + (int64_t)(r - t * heads) * a.d + c, s);
    }
}

}  // namespace

// A key tile's work grows with the group, and few key heads may leave SMs idle:
// the group's query heads are shared out to as many blocks (a divisor of the
// group) as give three items an SM.  Each then writes fp32 parts, read once more
// by k_attn_dkv_sum.  (5003 tokens, 14/2 heads of 64: gradients 109 us by one
// block a key tile and head, 84 us shared out.  8192 tokens, 32/8 heads of 128,
// 512 key tiles and heads: 1922 us by one block each, 1999 us shared out by two.)
int attn_dkv_splits(int64_t T, int rows, int Hkv, int group, int sms) {
    const int64_t items = (T + rows - 1) / rows * Hkv;
    for (int n = 1; n < group; ++n)
        if (group % n == 0 && items * n >= 3 * (int64_t)sms) return n;
    return group;
}

template <typename T> static cudaError_t launch_sum(const Ctx &c, const AttnArgs &a) {
    const int64_t n = 2 * a.T * a.Hkv * (a.d / 4), want = (n + 255) / 256, most = (int64_t)c.sms * 16;
    const dim3 grid((unsigned)(want < most ? want : most));
    return n + most * 256 < (int64_t)1 << 32 ? launch_pdl(k_attn_dkv_sum<T, uint32_t>, grid, dim3(256), 0, c.stream, a)
                                             : launch_pdl(k_attn_dkv_sum<T, int64_t>, grid, dim3(256), 0, c.stream, a);
}

cudaError_t launch_attn_dkv_sum(const Ctx &c, int dtype, const AttnArgs &a) {
    return dtype == DSC_BF16 ? launch_sum<bf16>(c, a) : launch_sum<float>(c, a);
}

// Every document's last tile may be partial; so may the two runs of rows that
// no document holds.  Offsets that go back and forth can ask for more tiles:
// then they count as no documents.
int64_t attn_max_tiles(int64_t T, int64_t n_docs, int rows) { return T / rows + n_docs + 2; }

size_t attn_list_bytes(int64_t T, int64_t n_docs, int rows) {
    return 16 + (size_t)attn_max_tiles(T, n_docs, rows) * sizeof(AttnTile);
}

cudaError_t launch_attn_tiles(const Ctx &c, const int32_t *cu, int64_t n_docs, int64_t T, int rows, size_t bytes,
                              void *rising, void *falling) {
    const int64_t most = T / rows + 1;
    int shift = 0;
    while ((most >> shift) >= NBIN) ++shift;
    return launch_pdl(k_attn_tiles, dim3(falling ? 2 : 1), dim3(1024), 0, c.stream, cu, (int)n_docs, (int)T, rows, shift,
                      bytes > (size_t)100 << 20 ? 1 : 0, (int)attn_max_tiles(T, n_docs, rows), static_cast<int *>(rising), static_cast<int *>(falling));
}

cudaError_t launch_attn_delta(const Ctx &c, int64_t T, int Hq, int d, const float *o, const float *dout, float *delta) {
    int L = 1;
    while (L < 32 && L * VecOf<float>::V < d) L <<= 1;
    const int64_t warps = (T * Hq + 4 * (32 / L) - 1) / (4 * (32 / L));
    const int64_t want = (warps + 7) / 8, most = (int64_t)c.sms * 8;
    return launch_pdl(k_attn_delta, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, c.stream, o, dout, delta, T, Hq,
                      d, L);
}

}  // namespace dsc
