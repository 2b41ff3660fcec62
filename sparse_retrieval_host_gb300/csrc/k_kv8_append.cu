// New rows into the paged 8-bit cache (kv8_append).
//
// Per (block, head): scale = 2^e with the smallest e for which
// amax <= 448 * 2^e, code = e4m3(x * 2^-e). Dividing by a power of two is exact,
// so the only rounding is e4m3's own; and when a later token makes a begun
// block's scale grow, the codes held are shifted by a power of two, which is
// exact too except where they fall into e4m3's subnormals.
//
// A unit is one (touched block, head, K or V): all new rows of the call that
// fall into that block, so nobody else writes the block's scale and no atomics
// are needed. Units are found from the requests' lengths by prefix sums that
// each CTA builds in shared memory. A value is read once (kept in registers
// between the maximum and the rounding) and written once: HBM-bound for
// prompts, latency for decode steps. A unit of up to 512 vectors of 8 values (16
// per lane) is done by one warp, eight to a CTA, without barriers; a larger one by
// the whole CTA (prompts of 10,000 rows x 8 heads x 128 in blocks of 32: 15 us by
// warps, 36 by CTAs; 4.5 TB/s against 6.8 measured for a copy).
#include "kv8_internal.cuh"

namespace srh {
namespace kv8 {
namespace {

constexpr int kThreads = 256;

struct Args {
    const uint16_t* x[2];       // K rows, V rows
    long long x_row[2];
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* table;
    const int32_t* len;
    const int32_t* cu;
    uint32_t* err;
    long long block_stride;
    int n_req, n_rows, heads, n_blocks, max_blocks;
    int bs_log2, dv_log2;       // log2 of block_tokens and of head_dim / 8
    int parts;                  // 1 (shared) or 2
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Magnitudes of bf16 values compare as unsigned 16-bit numbers, infinities and
// NaN on top: m = max(m, |pair|) in each half.
__device__ __forceinline__ uint32_t mag2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t mag8(uint32_t m, const uint4& w) {
    return mag2(mag2(mag2(mag2(m, w.x), w.y), w.z), w.w);
}
// A pair with 0 in place of values that are not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}
__device__ __forceinline__ uint4 finite8(const uint4& w) {
    return make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
}
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
    const float2 a = make_float2(bf_lo(w0) * inv, bf_hi(w0) * inv);
    const float2 b = make_float2(bf_lo(w1) * inv, bf_hi(w1) * inv);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
// The four e4m3 codes of a word times `f`, rounded to e4m3 again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(v.x * f, v.y * f), __NV_SATFINITE, __NV_E4M3);
        out |= c << (16 * i);
    }
    return out;
}

// GT threads per unit (32 or the CTA), NV vectors of 8 values kept in registers
// per thread; a unit with more reads the rest a second time (from L2).
template <int GT, int NV>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const __grid_constant__ Args a) {
    extern __shared__ int first[];      // [n_req + 1]: touched blocks before each request
    __shared__ long long warp_sums[33];
    __shared__ uint32_t warp_amax[kThreads / 32];
    const int tid = threadIdx.x;

    // touched blocks of each request: of up to 32 a lane each, in every warp;
    // of more by the whole CTA into shared memory
    const bool few = a.n_req <= 32;
    long long blocks = 0;
    bool bad = false;
    auto touched = [&](int b, int* q0, int* nq, int* len) -> int {
        *q0 = a.cu[b];
        *nq = a.cu[b + 1] - *q0;
        *len = a.len[b];
        if (*q0 < 0 || *nq < 0 || *nq > a.n_rows - *q0 || *len < *nq || *len > (a.max_blocks << a.bs_log2)) bad = true;
        else if (*nq > 0) return ((*len - 1) >> a.bs_log2) - ((*len - *nq) >> a.bs_log2) + 1;
        return 0;                       // (a request out of bounds is left out)
    };
    int my_q0 = 0, my_nq = 0, my_len = 0, my_first = 0;
    if (few) {
        const int b = tid & 31;
        const int n = b < a.n_req ? touched(b, &my_q0, &my_nq, &my_len) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (b >= o) incl += up;
        }
        my_first = incl - n;
        blocks = __shfl_sync(0xffffffffu, incl, 31);
    } else {
        for (int base = 0; base < a.n_req; base += kThreads) {
            const int b = base + tid;
            int q0, nq, len;
            const int n = b < a.n_req ? touched(b, &q0, &nq, &len) : 0;
            long long total;
            const long long incl = block_scan(n, warp_sums, &total);
            if (b < a.n_req) first[b] = (int)(blocks + incl - n);
            blocks += total;
        }
        if (tid == 0) first[a.n_req] = (int)blocks;
        __syncthreads();
    }
    // requests of an ascending cu touch no more blocks than there are rows; of a descending
    // one, which share rows, they may touch more than `first` counts
    const bool many = blocks > 0x7fffffffll;
    if (bad || many) atomicOr(a.err, kErrBounds);
    if (many) return;                                    // (every thread)

    const long long units = blocks * a.heads * a.parts;
    constexpr int kGroups = kThreads / GT;
    const int lane = tid % GT, group = tid / GT;
    bool odd = false;
    for (long long u0 = (long long)blockIdx.x * kGroups; u0 < units; u0 += (long long)gridDim.x * kGroups) {
        const long long u = u0 + group;
        if (u >= units) continue;           // whole groups
        const int h = (int)(u % a.heads);
        const long long r = u / a.heads;
        const int part = (int)(r % a.parts);
        const int blk = (int)(r / a.parts);
        int b, q0, nq, len, before;
        if (few) {
            // the last lane at or below blk (whole warps take part: a unit is a warp's or the CTA's)
            b = 31 - __clz(__ballot_sync(0xffffffffu, my_first <= blk && (tid & 31) < a.n_req));
            q0 = __shfl_sync(0xffffffffu, my_q0, b);
            nq = __shfl_sync(0xffffffffu, my_nq, b);
            len = __shfl_sync(0xffffffffu, my_len, b);
            before = __shfl_sync(0xffffffffu, my_first, b);
        } else {
            b = last_not_above(first, a.n_req, blk);
            q0 = a.cu[b];
            nq = a.cu[b + 1] - q0;
            len = a.len[b];
            before = first[b];
        }
        const int begin = len - nq;                                  // first new position
        const int j = (begin >> a.bs_log2) + blk - before;
        const int p0 = max(begin, j << a.bs_log2), p1 = min(len, (j + 1) << a.bs_log2);
        const int off = p0 - (j << a.bs_log2);                       // tokens the block held before
        const int id = a.table[(size_t)b * a.max_blocks + j];
        if (id < 0 || id >= a.n_blocks) {
            if (lane == 0) atomicOr(a.err, kErrBounds);
            continue;
        }
        const int nvec = (p1 - p0) << a.dv_log2;
        const uint16_t* x = a.x[part] + (size_t)(q0 + p0 - begin) * a.x_row[part] + ((size_t)h << (a.dv_log2 + 3));
        uint8_t* codes = a.codes[part] + (size_t)id * a.block_stride + (((size_t)h << a.bs_log2) << (a.dv_log2 + 3));
        float* sc = a.scale[part] + (size_t)id * a.heads + h;
        const float old = off ? *sc : 0.f;
        auto load = [&](int v) {
            const int row = v >> a.dv_log2, col = v & ((1 << a.dv_log2) - 1);
            return *reinterpret_cast<const uint4*>(x + (size_t)row * a.x_row[part] + col * 8);
        };

        uint4 keep[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * GT;
            keep[i] = v < nvec ? load(v) : make_uint4(0, 0, 0, 0);
        }
        // the group's largest magnitude, with or without what is not finite
        auto largest = [&](bool careful) -> uint32_t {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (careful) keep[i] = finite8(keep[i]);
                m = mag8(m, keep[i]);
            }
            for (int v = lane + NV * GT; v < nvec; v += GT) {
                const uint4 w = load(v);
                m = mag8(m, careful ? finite8(w) : w);
            }
            m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
            if (GT > 32) {                                  // the CTA
                if ((tid & 31) == 0) warp_amax[tid >> 5] = m;
                __syncthreads();
                m = warp_amax[0];
#pragma unroll
                for (int w = 1; w < kThreads / 32; ++w) m = max(m, warp_amax[w]);
                __syncthreads();
            }
            return m;
        };
        uint32_t amax = largest(false);
        const bool careful = amax >= 0x7f80u;               // the same for the whole group
        if (careful) {
            odd = true;
            amax = largest(true);
        }
        // bf16 bits -> the smallest e with amax <= 1.75 * 2^(e + 8)
        int e = (int)(amax >> 7) - 127 - ((amax & 0x7fu) <= 0x60u ? 8 : 7);
        if (e > kMaxExp) odd = true;
        e = min(max(e, kMinExp), kMaxExp);
        const float want = __uint_as_float((uint32_t)(e + 127) << 23);
        const float now = fmaxf(want, old);
        const float inv = 1.0f / now;
        if (now > old && off) {
            // the block's scale grows: codes of the tokens before
            const float f = old / now;
            const int words = off << (a.dv_log2 + 3 - 4);
            for (int i = lane; i < words; i += GT) {
                uint4* p = reinterpret_cast<uint4*>(codes) + i;
                uint4 w = *p;
                w.x = rescale4(w.x, f);
                w.y = rescale4(w.y, f);
                w.z = rescale4(w.z, f);
                w.w = rescale4(w.w, f);
                *p = w;
            }
        }
        uint8_t* dst = codes + ((size_t)off << (a.dv_log2 + 3));     // rows of a block are dense
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * GT;
            if (v < nvec)
                *reinterpret_cast<uint2*>(dst + (size_t)v * 8) =
                    make_uint2(codes4(keep[i].x, keep[i].y, inv), codes4(keep[i].z, keep[i].w, inv));
        }
        for (int v = lane + NV * GT; v < nvec; v += GT) {
            const uint4 raw = load(v), w = careful ? finite8(raw) : raw;
            *reinterpret_cast<uint2*>(dst + (size_t)v * 8) = make_uint2(codes4(w.x, w.y, inv), codes4(w.z, w.w, inv));
        }
        // every lane has read the old scale before its first shuffle / barrier above
        if (lane == 0) *sc = now;
    }
    if (odd) atomicOr(a.err, kErrRange);
}

}  // namespace

cudaError_t launch_append(const Cache& c, const kv8_pool& pool, const int32_t* table, const int32_t* len,
                          const int32_t* cu, int n_req, const uint16_t* k, long long k_row, const uint16_t* v,
                          long long v_row, int n_rows, cudaStream_t st) {
    Args a{};
    a.x[0] = k;
    a.x[1] = v;
    a.x_row[0] = k_row;
    a.x_row[1] = v_row;
    a.codes[0] = pool.k_codes;
    a.codes[1] = pool.v_codes;
    a.scale[0] = pool.k_scale;
    a.scale[1] = pool.v_scale;
    a.table = table;
    a.len = len;
    a.cu = cu;
    a.err = c.d_err;
    a.block_stride = c.block_stride;
    a.n_req = n_req;
    a.n_rows = n_rows;
    a.heads = c.cfg.n_kv_heads;
    a.n_blocks = c.cfg.n_blocks;
    a.max_blocks = c.cfg.max_blocks;
    a.bs_log2 = c.bs_log2;
    a.parts = c.cfg.shared_kv ? 1 : 2;
    a.dv_log2 = 4;
    while ((8 << a.dv_log2) < c.cfg.head_dim) ++a.dv_log2;
    // a request's n rows touch at most ceil(n / bs) + 1 blocks
    const long long most = ((long long)n_rows >> c.bs_log2) + 2ll * n_req;
    const long long units = (most < n_rows ? most : n_rows) * a.heads * a.parts;
    // threads for the vectors of an average unit: enough to hold them in registers (see the top)
    const long long blocks_lo = ((long long)n_rows + (1 << c.bs_log2) - 1) >> c.bs_log2;
    const long long rows_avg = n_rows / (blocks_lo > n_req ? blocks_lo : n_req);
    const long long vecs = rows_avg << a.dv_log2;
    const long long per = vecs <= 512 ? kThreads / 32 : 1;
    long long grid = (units + per - 1) / per;
    // no more CTAs of 16 vectors per lane than fit at once: each finds the units anew
    // (the prompts at the top 14.7 us, 15.4 with up to 8 per SM)
    const long long per_sm = vecs > 128 && vecs <= 512 ? 2 : 8;
    if (grid > per_sm * c.sm_count) grid = per_sm * c.sm_count;
    const size_t smem = (size_t)(n_req + 1) * sizeof(int);
    if (vecs <= 128) append_kernel<32, 4><<<(unsigned)grid, kThreads, smem, st>>>(a);
    else if (vecs <= 512) append_kernel<32, 16><<<(unsigned)grid, kThreads, smem, st>>>(a);
    else append_kernel<kThreads, 8><<<(unsigned)grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kv8
}  // namespace srh
