// Block tables and slot maps of the paged 8-bit cache, built on the GPU from
// request lengths (kv8_resize).
//
// With have_b = ceil(len_b / bs) and need_b = ceil(new_b / bs), request b gives
// back its table entries [need_b, have_b) or takes need_b - have_b blocks. Both
// are ranked by prefix sums over the requests, so the result does not depend on
// any order of execution:
//   released entry of rank i goes to free[top - 1 - i], top = n_free + released;
//   taken entry of rank k comes from free[top - 1 - k].
// Shrinking therefore undoes growing exactly, and a step that does both hands
// the released blocks on first.
//
// The work is a few loads per request and a store per changed entry, so the
// call is bound by latency. One CTA holds the three prefix sums in shared
// memory; ranks are spread over its threads, which find their request by
// bisection, so one long request costs no more than many short ones. Up to
// kInlineTokens new tokens it writes the positions and slots too (a second
// launch costs more than it saves); above, a second grid does.
#include "kv8_internal.cuh"

namespace srh {
namespace kv8 {
namespace {

constexpr int kThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kInlineTokens = 4096;

struct Args {
    const int32_t* new_len;
    int32_t* len;
    int32_t* table;
    int32_t* free_ids;
    int32_t* n_free;
    int32_t* cu;
    int32_t* pos;
    int64_t* slot;
    uint32_t* err;
    int n_req;
    int cap;
    int bs_log2;
    int n_blocks;
    int max_blocks;
    int fill_here;
};

// block_scan of three values at once.
__device__ __forceinline__ void block_scan3(long long& x, long long& y, long long& z, long long (*warp_sums)[33],
                                            long long* tx, long long* ty, long long* tz) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ux = __shfl_up_sync(0xffffffffu, x, o), uy = __shfl_up_sync(0xffffffffu, y, o),
                        uz = __shfl_up_sync(0xffffffffu, z, o);
        if (lane >= o) {
            x += ux;
            y += uy;
            z += uz;
        }
    }
    if (lane == 31) {
        warp_sums[0][warp] = x;
        warp_sums[1][warp] = y;
        warp_sums[2][warp] = z;
    }
    __syncthreads();
    if (warp < 3) {
        long long w = lane < nw ? warp_sums[warp][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        warp_sums[warp][lane] = w;
    }
    __syncthreads();
    if (warp > 0) {
        x += warp_sums[0][warp - 1];
        y += warp_sums[1][warp - 1];
        z += warp_sums[2][warp - 1];
    }
    *tx = warp_sums[0][nw - 1];
    *ty = warp_sums[1][nw - 1];
    *tz = warp_sums[2][nw - 1];
    __syncthreads();
}

// Position and slot of new token i (request b of the prefix sums cu, whose
// length after the call is new_len).
__device__ __forceinline__ void put_token(const Args& a, int i, int b, int begin, int count, int new_len) {
    const int p = new_len - count + (i - begin);
    const int id = a.table[(size_t)b * a.max_blocks + (p >> a.bs_log2)];
    a.pos[i] = p;
    a.slot[i] = ((int64_t)id << a.bs_log2) + (p & ((1 << a.bs_log2) - 1));
}

// A slot behind the last new token must not look like one: an earlier call's, or whatever
// a new array holds, becomes -1 (a negative one is left).
__device__ __forceinline__ void no_token(const Args& a, int i) {
    if (a.slot[i] >= 0) a.slot[i] = -1;
}

__global__ void __launch_bounds__(kThreads) resize_kernel(const Args a) {
    extern __shared__ int sums[];
    int* rel = sums;                    // [n_req + 1] released blocks before each request
    int* alc = rel + a.n_req + 1;       // taken blocks
    int* tok = alc + a.n_req + 1;       // new tokens
    int* kept = tok + a.n_req + 1;      // blocks that stay: min(have, need)
    __shared__ long long warp_sums[3][33];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int most = a.max_blocks << a.bs_log2;
    const int bs1 = (1 << a.bs_log2) - 1;

    long long R = 0, A = 0, N = 0;      // totals so far
    bool bad = false;
    for (int base = 0; base < a.n_req; base += nt) {
        const int b = base + tid;
        int r = 0, q = 0, t = 0, stay = 0;
        if (b < a.n_req) {
            const int was = a.len[b], will = a.new_len[b];
            if (was < 0 || was > most || will < 0 || will > most) {
                bad = true;
            } else {
                const int have = (was + bs1) >> a.bs_log2, need = (will + bs1) >> a.bs_log2;
                stay = min(have, need);
                r = max(0, have - need);
                q = max(0, need - have);
                t = max(0, will - was);
            }
        }
        long long tr, ta, tn, sr = r, sa = q, sn = t;
        block_scan3(sr, sa, sn, warp_sums, &tr, &ta, &tn);
        if (b < a.n_req) {
            // truncated only where a total makes the call fail below
            rel[b] = (int)(R + sr - r);
            alc[b] = (int)(A + sa - q);
            tok[b] = (int)(N + sn - t);
            kept[b] = stay;
        }
        R += tr;
        A += ta;
        N += tn;
    }
    const int depth = *a.n_free;
    if (depth < 0 || depth > a.n_blocks || R > a.n_blocks - depth || N > 0x7fffffffll) bad = true;
    if (a.pos && N > a.cap) bad = true;
    if (tid == 0) {
        rel[a.n_req] = (int)R;
        alc[a.n_req] = (int)A;
        tok[a.n_req] = (int)N;
    }
    bad = __syncthreads_or(bad);
    const bool none = !bad && A > depth + R;           // the same in every thread
    bad = bad || none;
    if (!bad) {
        // a released or taken entry that is no block fails the call before anything changes
        for (int i = tid; i < (int)R; i += nt) {
            const int b = last_not_above(rel, a.n_req, i);
            const int j = kept[b] + i - rel[b];
            const int id = a.table[(size_t)b * a.max_blocks + j];
            if (id < 0 || id >= a.n_blocks) bad = true;
        }
        // (the first R taken are the released ones)
#pragma unroll 4
        for (int k = (int)R + tid; k < (int)A; k += nt) {
            const int id = __ldcg(a.free_ids + depth + (int)R - 1 - k);
            if (id < 0 || id >= a.n_blocks) bad = true;
        }
        bad = __syncthreads_or(bad);
    }
    if (bad) {
        for (int b = tid; b <= a.n_req; b += nt) a.cu[b] = 0;
        if (tid == 0) atomicOr(a.err, none ? kErrNoBlocks : kErrBounds);
        if (a.pos && a.fill_here)
            for (int i = tid; i < a.cap; i += nt) no_token(a, i);
        return;
    }
    const int top = depth + (int)R;
    for (int i = tid; i < (int)R; i += nt) {
        const int b = last_not_above(rel, a.n_req, i);
        const int j = kept[b] + i - rel[b];
        int32_t* e = a.table + (size_t)b * a.max_blocks + j;
        a.free_ids[top - 1 - i] = *e;
        *e = -1;
    }
    __syncthreads();
#pragma unroll 4
    for (int k = tid; k < (int)A; k += nt) {
        const int b = last_not_above(alc, a.n_req, k);
        const int j = kept[b] + k - alc[b];
        // (the first ones written above by other threads, in L2)
        a.table[(size_t)b * a.max_blocks + j] = __ldcg(a.free_ids + top - 1 - k);
    }
    __syncthreads();
    for (int b = tid; b < a.n_req; b += nt) {
        a.len[b] = a.new_len[b];
        a.cu[b] = tok[b];
    }
    if (tid == 0) {
        a.cu[a.n_req] = (int)N;
        *a.n_free = top - (int)A;
    }
    if (!a.pos || !a.fill_here) return;
    for (int i = tid; i < (int)N; i += nt) {
        const int b = last_not_above(tok, a.n_req, i);
        put_token(a, i, b, tok[b], tok[b + 1] - tok[b], a.new_len[b]);
    }
    for (int i = (int)N + tid; i < a.cap; i += nt) no_token(a, i);
}

// Positions and slots of more than kInlineTokens tokens, after resize_kernel (which has
// left cu all 0 where it refused).
__global__ void __launch_bounds__(kFillThreads) fill_kernel(const Args a) {
    extern __shared__ int tok[];
    pdl_wait();
    const int N = a.cu[a.n_req];
    const int i = blockIdx.x * kFillThreads + threadIdx.x;
    if (i >= N && i < a.cap) no_token(a, i);
    if ((int)(blockIdx.x * kFillThreads) >= N) return;
    for (int b = threadIdx.x; b <= a.n_req; b += kFillThreads) tok[b] = a.cu[b];
    __syncthreads();
    if (i >= N) return;
    const int b = last_not_above(tok, a.n_req, i);
    put_token(a, i, b, tok[b], tok[b + 1] - tok[b], a.len[b]);
}

}  // namespace

cudaError_t set_resize_attrs() {
    return cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                4 * (kMaxBatch + 1) * (int)sizeof(int));
}

cudaError_t launch_resize(const Cache& c, const int32_t* new_len, int n_req, int32_t* len, int32_t* table,
                          int32_t* free_ids, int32_t* n_free, int32_t* cu, int32_t* pos, int64_t* slot, int cap,
                          cudaStream_t st) {
    Args a{};
    a.new_len = new_len;
    a.len = len;
    a.table = table;
    a.free_ids = free_ids;
    a.n_free = n_free;
    a.cu = cu;
    a.pos = pos;
    a.slot = slot;
    a.err = c.d_err;
    a.n_req = n_req;
    a.cap = cap;
    a.bs_log2 = c.bs_log2;
    a.n_blocks = c.cfg.n_blocks;
    a.max_blocks = c.cfg.max_blocks;
    a.fill_here = cap <= kInlineTokens;
    // enough threads for the requests and for the tokens written here, in whole warps
    int nt = 128;
    while (nt < kThreads && (nt < n_req || (a.fill_here && 2 * nt < cap))) nt *= 2;
    resize_kernel<<<1, nt, 4 * (n_req + 1) * sizeof(int), st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.fill_here || !pos) return e;
    return launch_k(fill_kernel, dim3((unsigned)((cap + (long long)kFillThreads - 1) / kFillThreads)), dim3(kFillThreads),
                    (n_req + 1) * sizeof(int), st, true, a);
}

}  // namespace kv8
}  // namespace srh
