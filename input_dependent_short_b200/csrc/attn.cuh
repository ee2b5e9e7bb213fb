// Shared pieces of the attention operators (include/dsc_attn.h): the kernel
// arguments, the tile list of packed documents, and the launch interface
// between the entry points (attn_api.cu) and the kernels.
#pragma once

#include <atomic>

#include "../../include/dsc_attn.h"
#include "kernels.cuh"

namespace dsc {

// One tile of consecutive rows of one document.  len < 0 marks rows that no
// document holds: rows [start, start - len) get zeros.
struct AttnTile {
    int start;  // the document's first row
    int len;    // its length
    int r0;     // the tile's first row inside the document
    int pad;
};

// A tile list in a workspace: 16 bytes with the number of tiles and a counter
// that starts at zero (persistent kernels draw items with it), then the tiles.
struct TileList {
    const int *count;
    int *next;
    const AttnTile *tiles;
};

// Short lists need no launch of their own: each block of the tensor-core
// kernels makes the list in its shared memory (at most this many tiles).
constexpr int INLINE_TILES = 64;

struct AttnArgs {
    int64_t T;
    int Hq, Hkv, d, group;
    int64_t qs, ks, vs;         // row strides of q, k, v (elements)
    int64_t dqs, dks, dvs;      // row strides of dq, dk, dv
    float scale;
    const void *q, *k, *v;
    void *o;                    // [T, Hq, d]
    float *lse;                 // [Hq, T]
    const void *dout;           // [T, Hq, d]
    float *delta;               // [Hq, T]: dout . o
    void *dq, *dk, *dv;
    // dk, dv summed over a group's query heads by nsplit blocks: their fp32 parts [nsplit][T, Hkv, d] (nsplit > 1)
    float *kpart, *vpart;
    int nsplit;
    TileList list;
    const int32_t *cu;  // not NULL: the list is short and made in the kernel from these offsets
    int n_docs;
};

// Raises a kernel's dynamic shared memory limit once per device (`done`: a bit per device, one word per kernel).
template <typename K> cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// attn_tiles.cu.  Tiles of `rows` rows: at most T / rows + n_docs + 2 of them,
// sorted by how many tiles of `rows` keys (the rising list) or of query rows
// (the falling one: the later tiles of a document have fewer) each has to
// visit, most first; by documents, the longest first, where the `bytes` of the
// inputs do not fit L2.
int64_t attn_max_tiles(int64_t T, int64_t n_docs, int rows);
size_t attn_list_bytes(int64_t T, int64_t n_docs, int rows);
// `falling` may be null: one list only.
cudaError_t launch_attn_tiles(const Ctx &c, const int32_t *cu, int64_t n_docs, int64_t T, int rows, size_t bytes,
                              void *rising, void *falling);
// delta[h][t] = dout[t][h] . o[t][h] (fp32; with bf16 the dq kernel forms it from the probabilities)
cudaError_t launch_attn_delta(const Ctx &c, int64_t T, int Hq, int d, const float *o, const float *dout, float *delta);

// Blocks that share a key tile's (of `rows` keys) group of query heads, and the sum of their parts.
int attn_dkv_splits(int64_t T, int rows, int Hkv, int group, int sms);
cudaError_t launch_attn_dkv_sum(const Ctx &c, int dtype, const AttnArgs &a);

// attn_simt.cu: the CUDA-core kernels (fp32)
constexpr int SIMT_ROWS = 32;
cudaError_t launch_attn_fwd_simt(const Ctx &c, const AttnArgs &a, int64_t max_tiles);
cudaError_t launch_attn_dq_simt(const Ctx &c, const AttnArgs &a, int64_t max_tiles);
cudaError_t launch_attn_dkv_simt(const Ctx &c, const AttnArgs &a, int64_t max_tiles);

// attn_tc_fwd.cu: the tensor-core kernel (bf16); tiles of attn_fwd_tc_rows(group) rows
int attn_fwd_tc_rows(int group);
cudaError_t launch_attn_fwd_tc(const Ctx &c, const AttnArgs &a, int64_t max_tiles);
int take_attn_fwd_status(cudaStream_t stream);
cudaError_t launch_feed_selftest(cudaStream_t stream);

// attn_tc_bwd.cu: the tensor-core gradients (bf16); tiles of ATTN_TC_BWD_ROWS rows
constexpr int ATTN_TC_BWD_ROWS = 128;
cudaError_t launch_attn_dkv_tc(const Ctx &c, const AttnArgs &a, int64_t max_tiles);
cudaError_t launch_attn_dq_tc(const Ctx &c, const AttnArgs &a, int64_t max_tiles);
int take_attn_bwd_status(cudaStream_t stream);

// attn_rope.cu
struct RopeArgs {
    int64_t T;
    int Hq, Hkv, d, rot;
    int64_t qs, ks, vs;
    float sign;                  // +1 forward, -1 gradient
    const int32_t *cu;           // NULL: row t belongs to sequence t
    int64_t n_seqs;
    const int32_t *seq_lens;     // NULL: positions are places inside the document
    const int32_t *table;
    int64_t n_pages, page, max_pages;
    const float *inv_freq;
    const void *q, *k, *v;
    void *q_out, *k_out, *k_cache, *v_cache;
};
cudaError_t launch_rope(const Ctx &c, int dtype, int interleaved, const RopeArgs &a);

// attn_decode.cu
struct DecodeArgs {
    int B, Hq, Hkv, d, group;
    int64_t qs;
    int64_t n_pages, max_pages;
    int page;
    float scale;
    const int32_t *seq_lens, *table;
    const void *q, *k, *v;
    void *o;
    float *lse;  // [B, Hq] or NULL
    float *part; // partial sums of segments that several blocks share
    int4 *rec;   // one record per block: the segment its share ends in
};
size_t decode_attn_ws_bytes(const Ctx &c, int dtype, int d);
cudaError_t launch_decode_attn(const Ctx &c, int dtype, DecodeArgs a, void *ws);

}  // namespace dsc
