// Rotary position rotation of q and k, its gradient, and the append to a
// paged key-value cache.
//
// One pass over the rows: each element is read once and written once, so the
// kernel is bound by memory (large calls) or by its launch (a decode step's
// few rows).  A block takes `TB` rows: their sequences and positions are found
// by one warp per row (a 32-way search of the offsets), the cosines and sines
// of a row's rot/2 angles are formed once for all of its heads, then threads
// move 16-byte vectors.
//
// The angle m * inv_freq is formed and reduced to half a turn in fp64 and only
// then given to the fp32 sine and cosine: at position 10^6 an fp32 product
// would be off by up to 0.03 radians, this way the error stays that of the
// fp32 functions.
#include "attn.cuh"

namespace dsc {
namespace {

constexpr int NTH = 128;
constexpr int TBMAX = NTH / 32;  // most rows of a block

struct RowInfo {
    int pos;            // position (valid when seq >= 0)
    int seq;            // -1: no sequence holds the row
    int64_t slot;       // element offset of (page, head 0, slot) in the caches, -1: none
};

// Sequences whose rows end at or before t: 32 probes at a time.
__device__ __forceinline__ int find_seq(const int32_t *cu, int n, int t, int lane) {
    int lo = 0, hi = n;  // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;  // asks whether sequence `at` ends at or before t
        const bool past = at < hi && cu[at + 1] <= t;
        const int c = __popc(__ballot_sync(FULL_MASK, past));  // offsets rise, so these are the first c probes
        if (c == 0) return lo;
        lo = lo + (c - 1) * step + 1;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

__device__ __forceinline__ RowInfo row_info(const RopeArgs &a, int64_t t, int lane) {
    RowInfo r{0, -1, -1};
    int s, first, count;
    if (a.cu) {
        s = find_seq(a.cu, (int)a.n_seqs, (int)t, lane);
        if (s >= a.n_seqs) return r;
        first = a.cu[s];
        count = a.cu[s + 1] - first;
        if (first < 0 || t < first || t >= (int64_t)first + count) return r;
    } else {
        s = (int)t;
        first = s;
        count = 1;
    }
    r.seq = s;
    r.pos = (int)t - first;
    if (a.seq_lens) {
        const int64_t pos = (int64_t)a.seq_lens[s] - count + r.pos;
        r.pos = (int)pos;
        if (pos >= 0 && pos < a.max_pages * a.page) {
            const int64_t pg = pos / a.page;
            const int page = a.table[(int64_t)s * a.max_pages + pg];
            if (page >= 0 && page < a.n_pages) r.slot = ((int64_t)page * a.Hkv * a.page + (pos - pg * a.page)) * a.d;
        }
    }
    return r;
}

// cos and sin of pos * f: whole turns are taken off in fp64, the rest is under half a turn
__device__ __forceinline__ float2 turn(int pos, float f, float sign) {
    double x = (double)pos * (double)f * 0.15915494309189533577;
    x -= rint(x);
    float s, c;
    sincospif((float)(2.0 * x), &s, &c);
    return make_float2(c, sign * s);
}

// One head of one row: where it comes from and goes.
template <typename T> struct HeadMove {
    const T *src;
    T *d0, *d1;   // destinations, either may be absent
    int r;        // row of the block
    bool rotate, zero;
};

template <typename T>
__device__ __forceinline__ HeadMove<T> head_move(const RopeArgs &a, const RowInfo *info, int64_t t0, int r, int h, int Hq) {
    HeadMove<T> m{nullptr, nullptr, nullptr, r, h < Hq + a.Hkv, false};
    const int64_t t = t0 + r;
    const RowInfo ri = info[r];
    m.zero = ri.seq < 0;
    if (h < Hq) {
        m.src = static_cast<const T *>(a.q) + t * a.qs + (int64_t)h * a.d;
        m.d0 = static_cast<T *>(a.q_out) + (t * a.Hq + h) * a.d;
        return m;
    }
    const int hk = m.rotate ? h - Hq : h - Hq - a.Hkv;
    m.src = (m.rotate ? static_cast<const T *>(a.k) + t * a.ks : static_cast<const T *>(a.v) + t * a.vs) + (int64_t)hk * a.d;
    if (m.rotate && a.k_out) m.d0 = static_cast<T *>(a.k_out) + (t * a.Hkv + hk) * a.d;
    if (ri.slot >= 0) m.d1 = static_cast<T *>(m.rotate ? a.k_cache : a.v_cache) + ri.slot + (int64_t)hk * a.page * a.d;
    return m;
}

// Whole vectors.  PAIRED: elements (i, i + rot/2) -- unit u < rot/2/V is the
// two vectors at u V and rot/2 + u V, the units behind are the plain vectors
// behind rot; else (2i, 2i+1) -- unit u is vector u.  A head takes 1 << HL
// threads; a thread has UNROLL units of different heads or rows in flight.
constexpr int UNROLL = 2;

template <typename T, bool PAIRED> __global__ void __launch_bounds__(NTH) k_rope(RopeArgs a, int TB, int HL) {
    constexpr int V = VecOf<T>::V;
    __shared__ __align__(16) float2 cs[TBMAX][64];  // cos, sin of a row's angles
    __shared__ RowInfo info[TBMAX];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * TB;
    const int nt = (int)min((int64_t)TB, a.T - t0);
    pdl_wait();
    pdl_trigger();
    if (warp < nt) {
        const RowInfo r = row_info(a, t0 + warp, lane);
        if (lane == 0) info[warp] = r;
    }
    __syncthreads();
    const int half = a.rot >> 1;
    for (int i = tid; i < nt * half; i += NTH) {
        const int r = i / half, j = i - r * half;
        cs[r][j] = turn(info[r].pos, a.inv_freq[j], a.sign);
    }
    __syncthreads();

    const int Hq = a.q ? a.Hq : 0, heads = Hq + a.Hkv + (a.v ? a.Hkv : 0);
    const int j = tid & ((1 << HL) - 1), step = NTH >> HL;
    const int pairs = PAIRED ? half / V : 0;
    const int units = PAIRED ? pairs + (a.d - a.rot) / V : a.d / V;
    for (int u = j; u < units; u += 1 << HL) {
        const bool two = PAIRED && u < pairs;
        const bool turned = PAIRED ? two : u * V < a.rot;
        const int c = PAIRED && !two ? a.rot + (u - pairs) * V : u * V;
        int r = 0, h = tid >> HL;
        while (h >= heads) {
            h -= heads;
            ++r;
        }
        while (r < nt) {
            HeadMove<T> m[UNROLL];
            uint4 x[UNROLL], y[UNROLL];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                m[k] = HeadMove<T>{nullptr, nullptr, nullptr, 0, false, false};
                x[k] = y[k] = make_uint4(0, 0, 0, 0);
                if (r < nt) {
                    m[k] = head_move<T>(a, info, t0, r, h, Hq);
                    if (!m[k].zero && (m[k].d0 || m[k].d1)) {
                        x[k] = ld16(m[k].src + c);
                        if (two) y[k] = ld16(m[k].src + c + half);
                    }
                    h += step;
                    while (h >= heads) {
                        h -= heads;
                        ++r;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                if (!m[k].d0 && !m[k].d1) continue;
                if (turned && m[k].rotate && !m[k].zero) {
                    const float4 *w4 = reinterpret_cast<const float4 *>(&cs[m[k].r][PAIRED ? c : c >> 1]);
                    if constexpr (PAIRED) {
                        float f[V], g[V], p[V], q[V];
                        unpack(x[k], f);
                        unpack(y[k], g);
#pragma unroll
                        for (int e = 0; e < V; e += 2) {
                            const float4 w = w4[e >> 1];  // cos, sin of two pairs
                            p[e] = f[e] * w.x - g[e] * w.y;
                            q[e] = f[e] * w.y + g[e] * w.x;
                            p[e + 1] = f[e + 1] * w.z - g[e + 1] * w.w;
                            q[e + 1] = f[e + 1] * w.w + g[e + 1] * w.z;
                        }
                        x[k] = pack(p);
                        y[k] = pack(q);
                    } else {
                        float f[V], p[V];
                        unpack(x[k], f);
#pragma unroll
                        for (int e = 0; e < V; e += 4) {
                            const float4 w = w4[e >> 2];
                            p[e] = f[e] * w.x - f[e + 1] * w.y;
                            p[e + 1] = f[e] * w.y + f[e + 1] * w.x;
                            p[e + 2] = f[e + 2] * w.z - f[e + 3] * w.w;
                            p[e + 3] = f[e + 2] * w.w + f[e + 3] * w.z;
                        }
                        x[k] = pack(p);
                    }
                }
                if (m[k].d0) {
                    st16(m[k].d0 + c, x[k]);
                    if (two) st16(m[k].d0 + c + half, y[k]);
                }
                if (m[k].d1) {
                    st16(m[k].d1 + c, x[k]);
                    if (two) st16(m[k].d1 + c + half, y[k]);
                }
            }
        }
    }
}

// Any rot: element by element (rot/2, or rot when interleaved, no multiple of a vector).
template <typename T> __global__ void __launch_bounds__(NTH) k_rope_any(RopeArgs a, int interleaved) {
    __shared__ float2 cs[64];
    __shared__ RowInfo info;
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (tid < 32) {
        const RowInfo r = row_info(a, t, tid);
        if (tid == 0) info = r;
    }
    __syncthreads();
    const int half = a.rot >> 1;
    for (int j = tid; j < half; j += NTH) cs[j] = turn(info.pos, a.inv_freq[j], a.sign);
    __syncthreads();
    const int Hq = a.q ? a.Hq : 0, heads = Hq + a.Hkv + (a.v ? a.Hkv : 0);
    for (int i = tid; i < heads * a.d; i += NTH) {
        const int h = i / a.d, u = i - h * a.d;
        const HeadMove<T> m = head_move<T>(a, &info, t, 0, h, Hq);
        if (!m.d0 && !m.d1) continue;
        float x = 0.f;
        if (!m.zero) {
            x = to_f<T>(m.src[u]);
            if (m.rotate && u < a.rot) {
                // element u is its pair's first (lead) or second; the partner lies at `o`
                const bool lead = interleaved ? !(u & 1) : u < half;
                const int p = interleaved ? u >> 1 : (lead ? u : u - half);
                const int o = interleaved ? u ^ 1 : (lead ? u + half : u - half);
                const float y = to_f<T>(m.src[o]);
                const float2 w = cs[p];
                x = lead ? x * w.x - y * w.y : y * w.y + x * w.x;
            }
        }
        const T out = from_f<T>(x);
        if (m.d0) m.d0[u] = out;
        if (m.d1) m.d1[u] = out;
    }
}

template <typename T> cudaError_t launch_t(const Ctx &c, int interleaved, const RopeArgs &a) {
    constexpr int V = VecOf<T>::V;
    const int half = a.rot >> 1;
    if (interleaved ? a.rot % V : half % V) return launch_pdl(k_rope_any<T>, dim3((unsigned)a.T), dim3(NTH), 0, c.stream, a, interleaved);
    const int units = interleaved ? a.d / V : half / V + (a.d - a.rot) / V;
    int HL = 0;
    while ((1 << HL) < units && HL < 5) ++HL;
    // enough blocks for four per SM first, then several rows a block (their angles and heads in one go)
    int TB = 1;
    while (TB < TBMAX && a.T / (TB * 2) >= 4 * c.sms) TB *= 2;
    const dim3 grid((unsigned)((a.T + TB - 1) / TB));
    return interleaved ? launch_pdl(k_rope<T, false>, grid, dim3(NTH), 0, c.stream, a, TB, HL)
                       : launch_pdl(k_rope<T, true>, grid, dim3(NTH), 0, c.stream, a, TB, HL);
}

}  // namespace

cudaError_t launch_rope(const Ctx &c, int dtype, int interleaved, const RopeArgs &a) {
    return dtype == DSC_BF16 ? launch_t<bf16>(c, interleaved, a) : launch_t<float>(c, interleaved, a);
}

}  // namespace dsc
