// Declarations shared by the paged 8-bit cache's translation units.
#pragma once

#include "srh_internal.cuh"

namespace srh {
namespace kv8 {

constexpr int kMaxBatch = 4096;     // requests of one call: their prefix sums fit shared memory
constexpr int kMinExp = -64;        // exponents of a block's scale
constexpr int kMaxExp = 64;

struct Cache {
    kv8_config cfg{};
    int device = 0;
    int sm_count = 0;
    int bs_log2 = 0;
    int d_blocks = 0;               // head_dim / 128
    long long block_stride = 0;     // bytes
    uint32_t* d_err = nullptr;
    float* d_part_o = nullptr;      // partial outputs of split attention items
    float* d_part_ml = nullptr;     // their maxima and sums
    int4* d_meta = nullptr;         // split items, by the chunk that they begin in
    int* d_ctrl = nullptr;          // the attention's chunk counter and count
    int* d_arrived = nullptr;       // parts of split items that are written (4-bit attention); zeros between calls
    size_t arrived_n = 0;
    size_t part_o_floats = 0;       // sizes of the three, which the launchers check
    size_t part_ml_floats = 0;
    size_t meta_n = 0;
    char last_error[256] = {0};
};

constexpr uint32_t kErrNoBlocks = 16u;   // error word bit: too few free blocks

// What the attention's scratch needs on a device with `sm_count` SMs.
void attend_scratch(int sm_count, int head_dim, size_t* o_floats, size_t* ml_floats, size_t* meta);
cudaError_t set_attend_attrs();
cudaError_t set_resize_attrs();

cudaError_t launch_resize(const Cache& c, const int32_t* new_len, int n_req, int32_t* len, int32_t* table,
                          int32_t* free_ids, int32_t* n_free, int32_t* cu, int32_t* pos, int64_t* slot, int cap,
                          cudaStream_t st);
cudaError_t launch_norm_rope(const Cache& c, const kv8_heads& q, const kv8_heads& k, int n_tok, int head_dim,
                             const int32_t* pos, long long pos_row, int n_axes, const uint8_t* axis,
                             const double* inv_freq, int rot_dim, int rot_off, int style, float eps, cudaStream_t st);
cudaError_t launch_append(const Cache& c, const kv8_pool& pool, const int32_t* table, const int32_t* len,
                          const int32_t* cu, int n_req, const uint16_t* k, long long k_row, const uint16_t* v,
                          long long v_row, int n_rows, cudaStream_t st);
cudaError_t launch_attend(const Cache& c, const kv8_pool& pool, const int32_t* table, const int32_t* len,
                          const int32_t* cu, int n_req, const uint16_t* q, long long q_row, int n_rows, int n_heads,
                          float scale, int window, uint16_t* out, long long out_row, cudaStream_t st);


// Rows of a 4-bit pool (bits 4) or of an 8-bit one (bits 8).
struct Part {
    uint8_t* codes;
    void* scale;
    uint16_t* x;                    // bf16 rows
    long long x_row;
};
struct Layer {
    Part part[2];                   // K, V
    int parts, bits;
    long long block_stride;
};
cudaError_t launch_append4(const Cache& c, const Layer& l, const int32_t* table, const int32_t* len, const int32_t* cu,
                           int n_req, int n_rows, cudaStream_t st);
cudaError_t launch_read(const Cache& c, const Layer& l, const int32_t* table, const int32_t* len, const int32_t* start,
                        const int32_t* cu, int n_req, int n_rows, cudaStream_t st);
// What kv4_attend needs of the scratch, and arrival counters.
void attend4_scratch(int sm_count, size_t* o_floats, size_t* ml_floats, size_t* meta, size_t* arrivals);
cudaError_t set_attend4_attrs();
cudaError_t launch_attend4(const Cache& c, const kv4_pool& pool, const int32_t* table, const int32_t* len,
                           const int32_t* cu, int n_req, const uint16_t* q, long long q_row, int n_rows, int n_heads,
                           float scale, int window, uint16_t* out, long long out_row, cudaStream_t st);

#ifdef __CUDACC__
// Inclusive sum over the CTA's threads (blockDim.x a multiple of 32, at most
// 1024) of a 64-bit value; `warp_sums` holds 33 entries; every thread gets the
// total too. Two barriers before and one after the last read of warp_sums.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
    *total = warp_sums[nw - 1];
    __syncthreads();
    return v;
}

// Last index b in [0, n) with first[b] <= i, for an ascending first[0..n) with
// first[0] <= i.
__device__ __forceinline__ int last_not_above(const int* first, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}
#endif

}  // namespace kv8
}  // namespace srh

struct kv8_cache : public srh::kv8::Cache {};
