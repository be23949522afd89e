// Paged KV cache: kernel parameter blocks and launch entry points (host side).
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "l2_params.h"

namespace l2 {

// Bits of a pool's status word (beside L2_DEV_ERR_BOUNDS): a call's index arrays or
// the bookkeeping they meet are not valid; the pool has too few free pages.
enum : int { L2_PAGES_ERR_ARGS = 4, L2_PAGES_ERR_FULL = 8 };

constexpr int kPagesMaxCall = 1024;  // sequences one call names
constexpr int kPagesThreads = 1024;  // threads of the one-block bookkeeping kernels

// Integers at the head of a pool's scratch: whether the last fork or free was refused (the kernel that copies its rows then does
// nothing), the pages a compaction moves, and whether the last extension was refused, which holds for the step's other
// layers too, whatever is called between them.  Then three lists of n_pages entries.
enum : int { kScrRefused = 0, kScrMoved = 1, kScrExtension = 2, kScrHead = 8 };

// A page pool.  Rows of head_size elements; strides in bytes.  Position p of sequence s is
// row p % page_size of page table[s * max_pages + p / page_size].
struct PagesView {
    char *k, *v;
    int *refs, *lens, *table, *err, *scratch;
    long long layer_stride, page_stride, head_stride, row_stride;  // bytes
    int n_layers, n_pages, n_kv_heads, page_size, n_seqs, max_pages;
    int row_bytes;  // head_size * element size, a multiple of 16
};

struct PagesAppend {
    char *k, *v;                                        // rows, read or written
    long long layer_stride, row_stride, head_stride;    // bytes
    const int *seqs, *starts;                           // [n], [n + 1] or nullptr (one row each)
    int n, rows, layer0, n_layers;
    bool extended;                                      // the call has just lengthened the sequences: their last pages are theirs
};

cudaError_t launch_pages_extend(const PagesView &p, int n, const int *seqs, const int *starts, int rows, cudaStream_t s);
// read: rows from the pool instead of into it.
cudaError_t launch_pages_rows(const PagesView &p, const PagesAppend &a, bool read, cudaStream_t s);
cudaError_t launch_pages_fork(const PagesView &p, int n, const int *src, const int *dst, const int *rows, cudaStream_t s);
cudaError_t launch_pages_free(const PagesView &p, int n, const int *seqs, bool compact, int num_sms, cudaStream_t s);

// Raises a kernel's shared-memory limit once per device (the attribute outlives the call).  least_regs: registers a thread it
// must have been compiled to, where it hands them around between its warps.
struct DeviceOnce {
    std::atomic<unsigned long long> done{0};
    cudaError_t smem(const void *fn, int bytes, int least_regs = 0) {
        int d = 0;
        cudaError_t e = cudaGetDevice(&d);
        if (e != cudaSuccess) return e;
        if (d < 64 && (done.load(std::memory_order_relaxed) >> d & 1)) return cudaSuccess;
        cudaFuncAttributes a{};
        if (least_regs && ((e = cudaFuncGetAttributes(&a, fn)) != cudaSuccess || a.numRegs < least_regs))
            return e != cudaSuccess ? e : cudaErrorInvalidDeviceFunction;
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && d < 64) done.fetch_or(1ull << d, std::memory_order_relaxed);
        return e;
    }
};

// Warps of a block of its kernels that walk, the last ones; with the tensor-core role there are four more before them.  (Which
// cost 0.7 us where nothing uses them: a call of 11.6 us took 12.3.)
constexpr int kWalkWarps = 8;
__host__ __device__ constexpr int walk_first(bool tc) { return tc ? 4 : 0; }
__host__ __device__ constexpr int attn_threads(bool tc) { return 32 * (walk_first(tc) + kWalkWarps); }

// Attention of one query row per sequence over its pages (attn_pages.cu).
struct PagesAttn {
    const char *k, *v;        // this layer's pages
    const int *lens, *table;
    int *err;
    long long page_stride, head_stride, row_stride;     // bytes
    const char *q;
    char *out;
    float *lse;               // [B][n_heads] natural-log sums, or nullptr
    long long q_row, q_head, o_row, o_head;             // bytes
    const int *seqs;          // [B] or nullptr (sequence b)
    const int *group_starts;  // [G + 1] or nullptr
    const int *prefix_lens;   // [G]
    int B, G, n_heads, n_kv_heads, head_size, page_size, max_pages, n_seqs, n_pages;
    int dtype, page_shift;    // log2(page_size), -1 where it is no power of two
    float scale_log2;         // scale * log2(e)
    // workspace
    int *plan;
    float *ws_ml, *ws_acc;
    int max_parts;            // parts the workspace holds
    int num_sms;              // blocks
    int tile_shift;           // log2 of the keys of a warp's tile
    bool tc;                  // prefixes may go to the tensor cores
    bool plan_in_block;       // every block plans for itself (no plan kernel before)
    bool wide;                // sequences as long as their tables would overflow the plan's 32 bits
    float *tc_ml, *tc_acc;    // its parts, by row
};

// Its kernels over 16-bit caches (attn_pages_16.cu) and fp32 caches (attn_pages_f32.cu): the logarithm of the keys of a
// warp's tile; whether 16-bit pages allow tensor-core tiles (fp32 pages all do).
int attn_pages_16_shift(int head_size);
bool attn_pages_tc_supported(const PagesAttn &p);
cudaError_t launch_attn_pages_16(const PagesAttn &p, cudaLaunchConfig_t cfg);
int attn_pages_f32_shift(int head_size);
cudaError_t launch_attn_pages_f32(const PagesAttn &p, cudaLaunchConfig_t cfg);

// cuTensorMapEncodeTiled, looked up once (l2_api.cu).
void *tensor_map_encoder();

size_t pages_attn_ws_bytes(int B, int G, int n_heads, int n_kv_heads, int head_size, int num_sms);
// Lays `p`'s workspace out in ws and launches the kernels.
cudaError_t launch_pages_attn(PagesAttn p, void *ws, int num_sms, cudaStream_t s);

}  // namespace l2
