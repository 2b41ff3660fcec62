// Rows into the 4-bit cache (kv4_append), and rows back from the 4-bit and the
// 8-bit one (kv4_read, kv8_read).
//
// In 4 bits a row of a head stands by itself: m = its smallest value (a bf16 value, so
// exact), s = bf16((largest - m) / 15), code = rint((x - m) / s). No later token
// changes what is held, unlike a scale shared by a block. Both ways are one read and one
// write of each value (append 2 + 0.5 bytes, read 0.5 + 2). Many rows take 1.5 (read) to 2.7 times (append) what their bytes
// would, as instructions bound them: 70 and 74 % of the issue slots; a few rows are latency.
//
// A CTA takes a range of rows. First a warp finds each row's request, by rounds of
// 32 samples of cu (two for 1,024 requests, against ten loads that wait for
// each other by bisection), and its block; then groups of lanes, 8 values to a lane, take
// the heads of all its rows in turn.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kv8_internal.cuh"

namespace srh {
namespace kv8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 32;            // of a CTA
constexpr uint32_t kLimit = 0x7b80u;    // bf16 bits of 2^120

struct Args {
    Part part[2];
    const int32_t* table;
    const int32_t* len;
    const int32_t* start;               // read: first token of each request
    const int32_t* cu;
    uint32_t* err;
    long long block_stride;
    int n_req, n_rows, heads, parts, n_blocks, max_blocks;
    int bs_log2;
    int rows;                           // per CTA
    uint32_t inv_row;                   // ceil(2^32 / units of a row): a unit's row by a product (0: one unit a row)
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Where the rows of a CTA lie: block (-1: none) and place in it.
struct Places {
    int block[kMaxRows];
    int at[kMaxRows];
};

// Row and place in it of unit u (below 2^14, of rows of at most 2^9 units: u inv_row / 2^32 exceeds the quotient
// by less than 2^-9).
__device__ __forceinline__ int row_of(const Args& a, int u) { return a.inv_row ? (int)__umulhi((uint32_t)u, a.inv_row) : u; }

// Fills in the places of rows [r0, r0 + n); false where cu descends (nothing is to be written).
template <bool READ>
__device__ __forceinline__ bool find_rows(const Args& a, int r0, int n, Places& p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long most = (long long)a.max_blocks << a.bs_log2;
    bool down = false, bad = false;
    auto out_of_bounds = [&](int c0, int c1, int l) {
        return c0 < 0 || c1 > a.n_rows || l < 0 || l > most || (!READ && l < (long long)c1 - c0);
    };
    // where request b's row r is, given its entries
    auto place = [&](int i, int r, int b, int c0, int c1, int l, int first) {
        int block = -1, at = 0;
        if (r >= c0 && r < c1 && l >= 0 && l <= most && (READ || (c0 >= 0 && c1 <= a.n_rows && l >= c1 - c0))) {
            const long long pos = READ ? (long long)first + (r - (long long)c0) : l - (c1 - r);
            if (pos >= 0 && pos < l) {
                block = a.table[(size_t)b * a.max_blocks + (pos >> a.bs_log2)];
                at = (int)pos & ((1 << a.bs_log2) - 1);
                if (block < 0 || block >= a.n_blocks) {
                    block = -1;
                    bad = true;
                }
            } else {
                bad = true;
            }
        }
        p.block[i] = block;
        p.at[i] = at;
    };
    if (a.n_req <= 32) {
        // a request per lane, a row per lane: two loads that wait for each other
        if (warp == 0) {
            const int b = min(lane, a.n_req - 1), c0 = a.cu[b], c1 = a.cu[b + 1], l = a.len[b], first = READ ? a.start[b] : 0;
            down = c1 < c0;
            if (blockIdx.x == 0 && out_of_bounds(c0, c1, l)) bad = true;
            // this lane's row: the last request that begins at or before it
            const int r = r0 + lane;
            int of = 0;
            for (int x = 1; x < a.n_req; ++x)
                if (__shfl_sync(0xffffffffu, c0, x) <= r) of = x;
            const int d0 = __shfl_sync(0xffffffffu, c0, of), d1 = __shfl_sync(0xffffffffu, c1, of);
            const int dl = __shfl_sync(0xffffffffu, l, of), df = __shfl_sync(0xffffffffu, first, of);
            if (lane < n) place(lane, r, of, d0, d1, dl, df);
        }
    } else {
        // every CTA looks cu over; the first reports requests that are left out
        for (int b = tid; b < a.n_req; b += kThreads) {
            const int c0 = a.cu[b], c1 = a.cu[b + 1];
            if (c1 < c0) down = true;
            if (blockIdx.x == 0 && out_of_bounds(c0, c1, a.len[b])) bad = true;
        }
        for (int i = warp; i < n; i += kWarps) {
            const int r = r0 + i;
            // the last request that begins at or before r: its number lies in [lo, hi)
            int lo = 0, hi = a.n_req;
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) >> 5;
                const int at = lo + lane * step;
                const bool before = at < hi && (lane == 0 || a.cu[at] <= r);
                const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
                lo += last * step;
                hi = min(hi, lo + step);
            }
            if (lane == 0) place(i, r, lo, a.cu[lo], a.cu[lo + 1], a.len[lo], READ ? a.start[lo] : 0);
        }
    }
    const bool stop = __syncthreads_or(down);
    if (bad || (stop && tid == 0)) atomicOr(a.err, kErrBounds);
    return !stop;
}

// The smallest and the largest of each half of two words, NaN where either is.
__device__ __forceinline__ uint32_t min2(uint32_t u, uint32_t v) {
    __nv_bfloat162 x, y;
    memcpy(&x, &u, 4);
    memcpy(&y, &v, 4);
    x = __hmin2_nan(x, y);
    memcpy(&u, &x, 4);
    return u;
}
__device__ __forceinline__ uint32_t max2(uint32_t u, uint32_t v) {
    __nv_bfloat162 x, y;
    memcpy(&x, &u, 4);
    memcpy(&y, &v, 4);
    x = __hmax2_nan(x, y);
    memcpy(&u, &x, 4);
    return u;
}
// bf16 bits: not finite -> 0, beyond 2^120 -> 2^120.
__device__ __forceinline__ uint32_t tame(uint32_t h) {
    if ((h & 0x7f80u) == 0x7f80u) return 0;
    return (h & 0x7fffu) > kLimit ? (h & 0x8000u) | kLimit : h;
}
__device__ __forceinline__ uint32_t tame2(uint32_t w) { return tame(w & 0xffffu) | tame(w >> 16) << 16; }

// The codes rint((x - m) / s) of 8 values, the division in fp32. With r = 1 / s and q = t r to nearest, q + r (t - q s) by
// two fused multiply-adds is t / s to nearest (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990: r is, and s has no mantissa of ones only): two operations a value more than the product
// alone, where divisions took 10 us of the prompts' 28, and products with divisions near halves as much.
__device__ __forceinline__ uint32_t codes8(const uint4& w, float m, float s) {
    constexpr float kRound = 12582912.f;    // 2^23 + 2^22: adding it rounds to an integer, in the low bits
    const float x[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y), bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
    uint32_t sum = 0;
    if (s >= 1e-30f && s <= 1e30f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const float t = x[i] - m, q = t * r;
            sum = sum * 16 + __float_as_uint(fmaf(fmaf(-q, s, t), r, q) + kRound);
        }
    } else {
        // (remainders and reciprocals might lose bits as subnormals; a scale that is one may leave quotients above 15)
#pragma unroll 1
        for (int i = 7; i >= 0; --i) {
            const float xi = i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : i == 3 ? x[3] : i == 4 ? x[4] : i == 5 ? x[5] : i == 6 ? x[6] : x[7];
            sum = sum * 16 + __float_as_uint(fminf(__fdiv_rn(xi - m, s), 15.f) + kRound);
        }
    }
    return sum - 0x4b400000u * 0x11111111u;  // each is 0x4b400000 more than its code
}

// LANES to a head, 8 values each; NV heads of a group are loaded before the first is used.
template <int LANES, int NV>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Args a) {
    constexpr int kGroups = kThreads / LANES, D = LANES * 8;
    __shared__ Places places;
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    const int r0 = blockIdx.x * a.rows, n = min(a.rows, a.n_rows - r0);
    const int per_row = a.heads * a.parts, units = n * per_row;
    bool odd = false;
    uint4 x[NV], next[NV];
    auto where = [&](int u, int* row, int* part, int* h) -> bool {
        *row = row_of(a, u);
        const int rest = u - *row * per_row;
        *part = rest >= a.heads;
        *h = rest - *part * a.heads;
        return u < units;
    };
    auto load = [&](int u0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int row, part, h;
            next[i] = make_uint4(0, 0, 0, 0);
            if (where(u0 + i * kGroups, &row, &part, &h))
                next[i] = __ldg(reinterpret_cast<const uint4*>(a.part[part].x + (size_t)(r0 + row) * a.part[part].x_row +
                                                               (size_t)h * D + lane * 8));
        }
    };
    load(group);                        // the values are on their way while their places are found
    if (!find_rows<false>(a, r0, n, places)) return;
    for (int u0 = group; u0 - group < units; u0 += kGroups * NV) {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = next[i];
        load(u0 + kGroups * NV);        // (nothing behind the last)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int row, part, h;
            const bool on = where(u0 + i * kGroups, &row, &part, &h) && places.block[row] >= 0;
            uint4& w = x[i];
            // the group's smallest value and its largest, negated, as the halves of one word
            auto reach = [&]() -> uint32_t {
                const uint32_t lo = min2(min2(w.x, w.y), min2(w.z, w.w)), hi = max2(max2(w.x, w.y), max2(w.z, w.w));
                uint32_t both = __byte_perm(min2(lo, lo >> 16), max2(hi, hi >> 16) ^ 0x8000u, 0x5410);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) both = min2(both, __shfl_xor_sync(0xffffffffu, both, o));
                return both;
            };
            uint32_t both = reach();
            // (magnitudes compare as integers, infinities and NaN on top)
            if (__any_sync(0xffffffffu, max(both & 0x7fffu, both >> 16 & 0x7fffu) > kLimit)) {
                const uint4 was = w;
                w = make_uint4(tame2(w.x), tame2(w.y), tame2(w.z), tame2(w.w));
                // (a row that belongs to no request may hold anything)
                if (on && (was.x != w.x || was.y != w.y || was.z != w.z || was.w != w.w)) odd = true;
                both = reach();
            }
            const float m = bf_lo(both), top = -bf_hi(both);
            const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(top - m, 15.f));
            const float s = __bfloat162float(sb);
            if (!on) continue;
            const uint32_t word = s > 0.f ? codes8(w, m, s) : 0;
            const size_t at = (size_t)h << a.bs_log2 | places.at[row];
            uint8_t* codes = a.part[part].codes + (size_t)places.block[row] * a.block_stride + at * (D / 2);
            *reinterpret_cast<uint32_t*>(codes + lane * 4) = word;
            if (lane == 0)
                reinterpret_cast<uint32_t*>(a.part[part].scale)[((size_t)places.block[row] * a.heads << a.bs_log2) + at] =
                    __bfloat16_as_ushort(sb) | __float_as_uint(m) >> 16 << 16;
        }
    }
    if (odd) atomicOr(a.err, kErrRange);
}

__device__ __forceinline__ uint32_t pack2(float u, float v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(u, v);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}

template <int LANES, int NV, int BITS>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ Args a) {
    constexpr int kGroups = kThreads / LANES, D = LANES * 8;
    __shared__ Places places;
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    const int r0 = blockIdx.x * a.rows, n = min(a.rows, a.n_rows - r0);
    if (!find_rows<true>(a, r0, n, places)) return;
    const int per_row = a.heads * a.parts, units = n * per_row;
    for (int u0 = group; u0 < units; u0 += kGroups * NV) {
        uint2 x[NV];
        float s[NV], m[NV];
        uint16_t* out[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = u0 + i * kGroups, row = row_of(a, u), rest = u - row * per_row;
            const int part = rest >= a.heads, h = rest - part * a.heads;
            out[i] = nullptr;
            if (u >= units || places.block[row] < 0) continue;
            const Part& p = a.part[part];
            const size_t at = (size_t)h << a.bs_log2 | places.at[row];
            const uint8_t* codes = p.codes + (size_t)places.block[row] * a.block_stride;
            out[i] = p.x + (size_t)(r0 + row) * p.x_row + (size_t)h * D + lane * 8;
            if (BITS == 4) {
                x[i].x = __ldg(reinterpret_cast<const uint32_t*>(codes + at * (D / 2)) + lane);
                const uint32_t sm = __ldg(reinterpret_cast<const uint32_t*>(p.scale) +
                                          ((size_t)places.block[row] * a.heads << a.bs_log2) + at);
                s[i] = bf_lo(sm);
                m[i] = bf_hi(sm);
            } else {
                x[i] = __ldg(reinterpret_cast<const uint2*>(codes + at * D) + lane);
                s[i] = __ldg(reinterpret_cast<const float*>(p.scale) + (size_t)places.block[row] * a.heads + h);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!out[i]) continue;
            float v[8];
            if (BITS == 4) {
                // (n s is exact in fp32: 4 and 8 significant bits; a code in the low bits of 2^23 is n more: a conversion
                // from integer would take four times as long)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = fmaf(__uint_as_float((x[i].x >> (4 * k) & 15u) | 0x4b000000u) - 8388608.f, s[i], m[i]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const uint32_t w = k < 4 ? x[i].x : x[i].y;
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (8 * (k & 2))), __NV_E4M3);
                    const float2 f = __half22float2(__half2(h));
                    v[k] = f.x * s[i];
                    v[k + 1] = f.y * s[i];
                }
            }
            *reinterpret_cast<uint4*>(out[i]) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        }
    }
}

Args args_of(const Cache& c, const Layer& l, const int32_t* table, const int32_t* len, const int32_t* start, const int32_t* cu,
             int n_req, int n_rows, unsigned* grid) {
    Args a{};
    a.part[0] = l.part[0];
    a.part[1] = l.part[1];
    a.table = table;
    a.len = len;
    a.start = start;
    a.cu = cu;
    a.err = c.d_err;
    a.block_stride = l.block_stride;
    a.n_req = n_req;
    a.n_rows = n_rows;
    a.heads = c.cfg.n_kv_heads;
    a.parts = l.parts;
    a.n_blocks = c.cfg.n_blocks;
    a.max_blocks = c.cfg.max_blocks;
    a.bs_log2 = c.bs_log2;
    // as few rows per CTA as give each thread four vectors, if there are CTAs enough
    const long long vecs = (long long)a.heads * a.parts * (c.cfg.head_dim / 8);
    long long rows = (8 * kThreads + vecs - 1) / vecs;
    const long long fill = ((long long)n_rows + 4 * c.sm_count - 1) / (4 * c.sm_count);
    if (rows > fill) rows = fill;
    a.rows = (int)(rows < 1 ? 1 : rows > kMaxRows ? kMaxRows : rows);
    const unsigned per_row = (unsigned)(a.heads * a.parts);
    a.inv_row = per_row == 1 ? 0 : (uint32_t)(((1ull << 32) + per_row - 1) / per_row);
    *grid = (unsigned)(((long long)n_rows + a.rows - 1) / a.rows);
    return a;
}

}  // namespace

cudaError_t launch_append4(const Cache& c, const Layer& l, const int32_t* table, const int32_t* len, const int32_t* cu,
                           int n_req, int n_rows, cudaStream_t st) {
    unsigned grid;
    const Args a = args_of(c, l, table, len, nullptr, cu, n_req, n_rows, &grid);
    if (c.cfg.head_dim == 128) append_kernel<16, 2><<<grid, kThreads, 0, st>>>(a);
    else append_kernel<32, 2><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_read(const Cache& c, const Layer& l, const int32_t* table, const int32_t* len, const int32_t* start,
                        const int32_t* cu, int n_req, int n_rows, cudaStream_t st) {
    unsigned grid;
    const Args a = args_of(c, l, table, len, start, cu, n_req, n_rows, &grid);
    if (l.bits == 4) {
        if (c.cfg.head_dim == 128) read_kernel<16, 4, 4><<<grid, kThreads, 0, st>>>(a);
        else read_kernel<32, 4, 4><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (c.cfg.head_dim == 128) read_kernel<16, 4, 8><<<grid, kThreads, 0, st>>>(a);
        else if (c.cfg.head_dim == 256) read_kernel<32, 4, 8><<<grid, kThreads, 0, st>>>(a);
        else read_kernel<64, 4, 8><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kv8
}  // namespace srh
