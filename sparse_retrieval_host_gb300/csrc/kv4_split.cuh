// How the 4-bit attention's kernels cut their work: found on the device from the
// lengths, so that a captured call follows new ones.
//
// A row tile is RT of the (token, head) rows that share a KV head of a request. Row tiles k and
// nrt - 1 - k of a causal request together see about as many tokens whatever k is: pairs of them are
// items of equal work, P units each, in the order (request, KV head, pair, units of the later row
// tile, then of the earlier, then nothing). A unit is a tile of 128 tokens, or half of one
// where a row tile is more than half full (HALVES: the matrix products of the other half of its rows);
// SW units before a row tile's first stand for what its start and end cost.
// The U units are cut into chunks of equal numbers, one per CTA. A row tile whose units fall
// into several chunks leaves partial sums, which are joined in chunk order: of few rows by the last CTA to write its part
// (finish), of many by a kernel of their own.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv8_internal.cuh"

namespace srh {
namespace kv8 {
namespace split {

constexpr int kTile = 128;               // tokens
constexpr int kMaxUnits = 1 << 30;
// Units of a chunk at least, of large row tiles: seven prompts of 58 tokens 26.0 us with 1, 22.9 with 4, 21.7 with 10, but two
// of 556 tokens on 2,384 34.2, 34.4, 36.9.
constexpr int kLeast = 4;

// What every kernel is given.
struct Args {
    const uint16_t* q;
    uint16_t* out;
    long long q_row, out_row, block_stride;
    const int32_t* cu;
    const int32_t* len;
    const int32_t* table;
    const uint8_t* kc;
    const uint8_t* vc;
    const uint32_t* ks;                          // (scale, minimum), bf16 each
    const uint32_t* vs;
    float* part_o;
    float* part_ml;
    int* arrived;                                // [3][arrived_n], zeros between calls
    int arrived_n;                               // CTAs at most
    int4* meta;                                  // split row tiles by the chunk that they begin in, for the join: (parts |
                                                 // rows << 12, first row of q and out, row, KV head)
    int* ctrl;                                   // [1]: chunks of this call
    uint32_t* err;
    int n_req, n_rows, kv_heads, group;          // group = query heads / kv_heads
    unsigned long long per_group;                // ceil(2^64 / group); 0 for a group of 1
    int rows_lo, rows_hi;                        // takes requests of rows_lo < rows <= rows_hi per KV head
    int bs_log2, n_blocks, max_blocks;
    float scale_log2;
    int window;                                  // 0: none
};

struct Request {
    int q0, nq, len;
    int nrt;           // row tiles
    int pairs;         // of row tiles, per KV head
    int P;             // units of a pair: at least what its two row tiles take
};

// x / group for 0 <= x < 2^32: with m = ceil(2^64 / group), x m / 2^64 exceeds x / group
// by less than x / 2^64, which is less than the 1 / group up to the next integer.
__device__ __forceinline__ int by_group(const Args& a, int x) {
    return a.group == 1 ? x : (int)__umul64hi((unsigned long long)(uint32_t)x, a.per_group);
}

// Token tiles that any row of row tile rt sees, from *first on (0: none; it has its zeros to write).
template <int RT>
__device__ __forceinline__ int tiles_of(const Args& a, const Request& r, int rt, int* first) {
    const int c = r.len - r.nq;                                    // position of the first query
    const int p_lo = c + by_group(a, rt * RT), p_hi = c + min(r.nq - 1, by_group(a, (rt + 1) * RT - 1));
    *first = a.window ? max(0, p_lo - a.window + 1) / kTile : 0;
    return max(0, (p_hi < 0 ? 0 : p_hi / kTile + 1) - *first);
}
template <int RT, bool HALVES>
__device__ __forceinline__ int weight(const Args& a, const Request& r, int rt) {
    return HALVES && r.nq * a.group - rt * RT > RT / 2 ? 2 : 1;
}
template <int RT, bool HALVES, int SW>
__device__ __forceinline__ int units_of(const Args& a, const Request& r, int rt) {
    int first;
    return max(1, tiles_of<RT>(a, r, rt, &first)) * weight<RT, HALVES>(a, r, rt) + SW;
}

template <int RT, bool HALVES, int SW>
__device__ __forceinline__ Request request(const Args& a, int b, bool* bad) {
    Request r;
    const int c0 = a.cu[b], c1 = a.cu[b + 1], n = a.len[b], most = a.max_blocks << a.bs_log2;
    r.q0 = min(max(c0, 0), a.n_rows);
    r.nq = min(max(c1, r.q0), a.n_rows) - r.q0;               // (rows outside q are not there)
    r.len = n;
    if (c0 != r.q0 || c1 != r.q0 + r.nq) *bad = true;
    if (n < 0 || n > most) {                                  // no such request
        *bad = true;
        r.nq = r.len = 0;
    }
    const int rows = r.nq * a.group;
    r.nrt = rows > a.rows_lo && rows <= a.rows_hi ? (rows + RT - 1) / RT : 0;
    r.pairs = (r.nrt + 1) >> 1;
    r.P = 0;
    if (r.nrt == 0) return r;
    constexpr int W = HALVES ? 2 : 1;
    const int c = r.len - r.nq, all = max(1, (r.len + kTile - 1) / kTile);
    if (r.nrt <= 2) {
        r.P = units_of<RT, HALVES, SW>(a, r, 0) + (r.nrt == 2 ? units_of<RT, HALVES, SW>(a, r, 1) : 0);
    } else if (a.window || c < 0) {
        r.P = 2 * W * (int)min((long long)all, ((long long)(a.window ? a.window : all * kTile) + RT / a.group + 1) / kTile + 2) + 2 * SW;
    } else {
        // positions of the last rows of k and nrt - 1 - k add up to those of 0 and of a full last row
        // tile, or one more: so do their tiles
        r.P = W * ((c + (RT - 1) / a.group) / kTile + (c + (int)(((long long)r.nrt * RT - 1) / a.group)) / kTile + 3) + 2 * SW;
    }
    return r;
}

// A chunk's share of one row tile.
struct Segment {
    int b, h, row0, nr;      // rows of the row tile in the request's (token, head) order
    int q0, nq, len;
    int p_lo, p_hi;          // positions of the first and the last row
    int t0, n;               // first token tile, and tiles to run (0: no row sees any)
    int v0, parts, part;     // the chunk in which the row tile begins, chunks that share it, this one's place
};

struct Chunks {
    int n, base, rem;
    __device__ __forceinline__ int begin(int v) const { return v * base + min(v, rem); }
    __device__ __forceinline__ int of(int u) const {
        return u < rem * (base + 1) ? u / (base + 1) : rem + (u - rem * (base + 1)) / base;
    }
};

// The units before each request into `first`, by all T threads of the CTA; false where this CTA has
// nothing to do. `warp_sums` as for block_scan.
template <int RT, bool HALVES, int SW, int T>
__device__ __forceinline__ bool count(const Args& a, int* first, long long* warp_sums, Chunks* ch) {
    const int tid = threadIdx.x;
    bool bad = false, stop = false;
    long long U = 0;
    for (int base = 0; base < a.n_req; base += T) {
        const int b = base + tid;
        long long mine = 0, total;
        if (b < a.n_req) {
            const Request r = request<RT, HALVES, SW>(a, b, &bad);
            mine = (long long)r.pairs * r.P * a.kv_heads;
            if (a.cu[b + 1] < a.cu[b]) stop = true;           // requests may share rows
        }
        const long long incl = block_scan(mine, warp_sums, &total);
        if (b < a.n_req) first[b] = (int)(U + incl - mine);
        U += total;
    }
    stop = __syncthreads_or(stop) || U > kMaxUnits;
    if (blockIdx.x == 0 && (bad || (stop && tid == 0))) atomicOr(a.err, kErrBounds);
    if (stop || U == 0) return false;
    const int n_grid = gridDim.x, most = max(RT >= 128 ? kLeast : 1, ((int)U + n_grid - 1) / n_grid);
    ch->n = ((int)U + most - 1) / most;                       // as few as keep the largest share the same
    ch->base = (int)U / ch->n;
    ch->rem = (int)U - ch->base * ch->n;
    return (int)blockIdx.x < ch->n;
}

// The segment at unit *u of chunk v (which ends at u1); moves *u on. False: none there.
template <int RT, bool HALVES, int SW>
__device__ __forceinline__ bool next_segment(const Args& a, const int* first, const Chunks& ch, int v, int* u, int u1, Segment* s) {
    while (*u < u1) {
        bool bad = false;                                     // (reported by count)
        s->b = last_not_above(first, a.n_req, *u);
        const Request r = request<RT, HALVES, SW>(a, s->b, &bad);
        const int in = *u - first[s->b], pair = in / r.P, o = in - pair * r.P;
        s->h = pair / r.pairs;
        const int k = pair - s->h * r.pairs, late = r.nrt - 1 - k;
        const int n_late = units_of<RT, HALVES, SW>(a, r, late);
        int rt = late, at = o, n = n_late;
        if (o >= n_late) {
            rt = k;
            at = o - n_late;
            n = k < late ? units_of<RT, HALVES, SW>(a, r, k) : 0;
        }
        if (at >= n) {                                        // what a pair has too many
            *u += min(r.P - o, u1 - *u);
            continue;
        }
        // its first SW units stand for its start and end: chunks that only have some of those have no part
        const int take = min(n - at, u1 - *u), u_rt = *u - at;
        *u += take;
        if (at + take <= SW) continue;
        s->row0 = rt * RT;
        s->nr = min(RT, r.nq * a.group - s->row0);
        s->q0 = r.q0;
        s->nq = r.nq;
        s->len = r.len;
        s->p_lo = r.len - r.nq + by_group(a, s->row0);
        s->p_hi = r.len - r.nq + by_group(a, s->row0 + s->nr - 1);
        s->v0 = ch.of(u_rt + SW);
        s->parts = ch.of(u_rt + n - 1) - s->v0 + 1;
        s->part = v - s->v0;
        int t_first;
        const int W = weight<RT, HALVES>(a, r, rt), tiles = tiles_of<RT>(a, r, rt, &t_first);
        const int from = max(0, at - SW), to = at + take - SW;
        const int lo = min(tiles, (from + W - 1) / W), hi = min(tiles, (to + W - 1) / W);
        s->t0 = t_first + lo;
        s->n = hi - lo;
        return true;
    }
    return false;
}

// Where part i of a row tile that begins in chunk v0 leaves its sums: a chunk's last row
// tile, or its first.
__device__ __forceinline__ size_t slot_of(int v0, int i) { return (size_t)(2 * (v0 + i) + (i == 0)); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Pairs of fp32 values in one 64-bit register (one instruction for both).
using u64 = unsigned long long;
__device__ __forceinline__ u64 pack(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(u64 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}

constexpr float kLow = -1e30f;           // reference of a row that has seen no token

// Parts i0, i0 + step, .. (cnt of them) of a row tile together, by threads tid of T: part i has
// reference m_i, sum l_i and outputs O_i of each row, and sum 2^(m_i - m) O_i, sum 2^(m_i - m) l_i, in order,
// become `out` (FINAL) or part i0. All T threads of the CTA take part.
template <int RT, int D, bool FINAL>
__device__ __forceinline__ void join(const Args& a, const Segment& s, int i0, int step, int cnt, int tid, int T) {
    float2* const ml = reinterpret_cast<float2*>(a.part_ml);
    // rows of one thread at most, so that a part's statistics are read before they are written
    for (int x0 = 0; x0 < s.nr * (D / 4); x0 += T) {
        const int x = x0 + tid, row = x / (D / 4), d = (x - row * (D / 4)) * 4;
        const bool on = row < s.nr;
        float m = kLow, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
#pragma unroll 8
            for (int i = 0; i < cnt; ++i) {
                const float2 st = __ldcg(&ml[slot_of(s.v0, i0 + i * step) * RT + row]);
                if (st.y != 0.f) m = fmaxf(m, st.x);
            }
#pragma unroll 8
            for (int i = 0; i < cnt; ++i) {
                const size_t at = slot_of(s.v0, i0 + i * step) * RT + row;
                const float2 st = __ldcg(&ml[at]);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + d));
                if (st.y == 0.f) continue;                    // a part with no weight does not count
                const float f = ex2(st.x - m);
                sum = fmaf(f, st.y, sum);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
        }
        if (FINAL) {
            if (!on) continue;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int rr = s.row0 + row, tok = by_group(a, rr);
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            uint2 w;
            memcpy(&w.x, &lo, 4);
            memcpy(&w.y, &hi, 4);
            *reinterpret_cast<uint2*>(a.out + (size_t)(s.q0 + tok) * a.out_row + (size_t)(s.h * a.group + rr - tok * a.group) * D + d) = w;
        } else {
            const size_t at = slot_of(s.v0, i0) * RT + row;
            __syncthreads();
            if (!on) continue;
            *reinterpret_cast<float4*>(a.part_o + at * D + d) = acc;
            if (d == 0) ml[at] = make_float2(m, sum);
        }
    }
}

// After a part's sums are written and the threads that wrote them have met: the last of up to kFan
// neighbours to get here joins them, the last group of neighbours the groups (parts of one long request
// are as many as CTAs, and one SM would read them for longer than they took). Counters: of a row tile's
// first group by its chunk, of the others by theirs, and of its groups; back to zero for the next call.
// All T threads of the CTA take part.
constexpr int kFan = 12;
template <int RT, int D>
__device__ __forceinline__ void finish(const Args& a, const Segment& s, int tid, int T, volatile int* flag) {
    const int k = s.part / kFan, i0 = k * kFan, cnt = min(kFan, s.parts - i0), groups = (s.parts + kFan - 1) / kFan;
    auto last_of = [&](int* counter, int n) -> bool {         // this CTA is the last
        if (tid == 0) {
            __threadfence();                                  // (what this thread has seen written is ordered with it)
            const bool last = atomicAdd(counter, 1) == n - 1;
            if (last) *counter = 0;
            __threadfence();
            *flag = last;
        }
        __syncthreads();
        return *flag;
    };
    if (!last_of(a.arrived + (k == 0 ? s.v0 : a.arrived_n + s.v0 + i0), cnt)) return;
    if (groups == 1) {
        join<RT, D, true>(a, s, i0, 1, cnt, tid, T);
        return;
    }
    join<RT, D, false>(a, s, i0, 1, cnt, tid, T);
    __syncthreads();
    if (last_of(a.arrived + 2 * a.arrived_n + s.v0, groups)) join<RT, D, true>(a, s, 0, kFan, groups, tid, T);
}

}  // namespace split

// The kernel of many rows per KV head: its share of the handle's scratch (the first), and its launch, which leaves it to the
// caller to check that it is there.
void chunk4_scratch(int sm_count, size_t* o_floats, size_t* ml_floats, size_t* meta);
cudaError_t set_chunk4_attrs();
cudaError_t launch_chunk4(int sm_count, int head_dim, const split::Args& a, cudaStream_t st);
// .. and of what joins its parts, after the kernel of few rows that runs beside it.
cudaError_t launch_join4(int sm_count, int head_dim, const split::Args& a, cudaStream_t st);

}  // namespace kv8
}  // namespace srh
