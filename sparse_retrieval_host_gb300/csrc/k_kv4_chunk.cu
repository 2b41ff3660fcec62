// Attention over the paged 4-bit cache (kv4_attend) for requests of many query rows per KV head
// (prompt chunks, drafts of wide groups): 128-dim heads on the 5th-generation tensor cores.
//
// Rows are the M dimension of both products, S = Q K^T and O = P V. Codes become fp16 values in
// shared memory once per tile of 128 tokens and are used by up to 256 rows:
//   k = (m + n s) 2^(14 - e), e the exponent of the tile's largest magnitude,
// one rounding of 2^-12 per value (or 2^-40 of the tile's largest); the power of two goes into
// the scores' factor, V's into the exponent u = score + e of the weights 2^(u - ref), which are rounded to
// fp16, and is taken out of the softmax's sums again. A thread holds a row, so maxima and sums
// need no exchange; a row's reference moves only when a weight would pass 2^15.5.
//
// A CTA runs two lanes of 128 rows, each with its own S and O in TMEM (P lies over S), so that one
// lane's exponentials run beside the other's products. Of a row tile of more than 128 rows the lanes
// take the two halves, tile by tile of the same tokens; of one of up to 128 rows they take the same
// rows and every other tile, and add up at the end.
//
// Per 128 tokens x 256 rows: 2,048 cycles of MMA at the fp16 rate, 2,048 of exponentials (16 a cycle),
// 2,048 of shared memory (QK reads both operands: 1,024; PV one: 512; expanding writes 512): no unit
// is free, the floor of one is that of all.
//
// Roles: warps 0-3 and 4-7 softmax of the two lanes, 8-11 expand K, 12-15 V (a thread a token, the
// next tile's codes in registers), 16 issues the MMAs. All waits are on mbarriers and bounded.
#include "kv4_split.cuh"
#include "umma.cuh"

namespace srh {
namespace kv8 {
namespace {

using namespace umma;
using namespace split;

constexpr int kRT = 256, kD = 128;
constexpr int kThreads = 17 * 32;
constexpr int kHalf = 16384;             // 128 rows of 64 fp16 values
constexpr int kTileBytes = 2 * kHalf;
constexpr int kOffK = 2 * kTileBytes;    // behind Q of the two lanes
constexpr int kOffV = kOffK + 2 * kTileBytes;
constexpr int kOffBars = kOffV + 2 * kTileBytes;
constexpr int kInfo = 4;                 // tiles whose exponents are held
constexpr float kHead = 10.f;            // log2 of the weight that a new reference gives a row's maximum
constexpr float kRoom = 15.5f;           // a row's reference moves when a weight would pass 2^15.5
constexpr int kTop = 14;                 // exponent of the largest fp16 value of a tile, and of a row of Q

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t k_info[kInfo], v_info[kInfo];   // a tile's exponent (and which tokens there are) is written
    uint64_t max_in[2];                  // K's / V's warps have given a tile's maxima
    uint64_t s_full[2], p_full[2];       // of each lane: scores are in TMEM, weights are
    uint64_t q_full, o_full;             // queries are in shared memory; outputs are complete
    uint64_t met[2];                     // the softmax warps meet
    uint64_t drain;
    long long warp_sums[33];
    uint32_t tmem_base;
    int abort, last;
    uint32_t most[2][2][4];              // [K, V][tile & 1][warp]: largest magnitude
    alignas(16) uint32_t there[kInfo][4];            // tokens that exist, a bit each
    float k_factor[kInfo];               // 2^(e - 14)
    int v_exp[kInfo];                    // e
    float2 stat[2][128];                 // reference and sum of each lane's rows
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
// D += A B with A (fp16, two to a column) in TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return h;
}
__device__ __forceinline__ uint32_t bits(__half2 h) {
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The eight values of a word of codes, as pairs (i, i + 4). A code in the low bits of 1024 is
// exact there; without the 1024 it is n, or 16 n.
__device__ __forceinline__ uint4 values8(uint32_t w, __half2 s, __half2 s16, __half2 m) {
    const __half2 k = __float2half2_rn(1024.f);
    const uint32_t x = w >> 8;
    uint4 r;
    r.x = bits(__hfma2(__hsub2(as_half2((w & 0x000f000fu) | 0x64006400u), k), s, m));
    r.y = bits(__hfma2(__hsub2(as_half2((w & 0x00f000f0u) | 0x64006400u), k), s16, m));
    r.z = bits(__hfma2(__hsub2(as_half2((x & 0x000f000fu) | 0x64006400u), k), s, m));
    r.w = bits(__hfma2(__hsub2(as_half2((x & 0x00f000f0u) | 0x64006400u), k), s16, m));
    return r;
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}

__global__ void __launch_bounds__(kThreads, 1) chunk4_kernel(const __grid_constant__ Args a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Bars& bs = *reinterpret_cast<Bars*>(sm + kOffBars);
    int* const first = reinterpret_cast<int*>(sm + kOffBars + sizeof(Bars));
    volatile int* abort = &bs.abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_trigger();                       // (the kernel of few rows, which reads nothing of this one)
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bs.k_full[i], 4);
            mbar_init(&bs.k_empty[i], 1);
            mbar_init(&bs.v_full[i], 4);
            mbar_init(&bs.v_empty[i], 1);
            mbar_init(&bs.max_in[i], 4);
            mbar_init(&bs.s_full[i], 1);
            mbar_init(&bs.p_full[i], 4);
            mbar_init(&bs.met[i], 8);
        }
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(&bs.k_info[i], 4);
            mbar_init(&bs.v_info[i], 4);
        }
        mbar_init(&bs.q_full, 8);
        mbar_init(&bs.o_full, 1);
        mbar_init(&bs.drain, 1);
        bs.abort = 0;
        fence_mbar_init();
    }
    Chunks ch;
    if (!count<kRT, true, kThreads>(a, first, bs.warp_sums, &ch)) return;      // every thread
    if (warp == 16) tmem_alloc(&bs.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bs.tmem_base;                        // S of the lanes at 0 and 128, O at 256 and 384
    const int cta = blockIdx.x;
    int u = ch.begin(cta);
    const int u1 = ch.begin(cta + 1);
    bool ok = true;
    Segment s;
    uint32_t G = 0;                                            // tiles before this segment
    // (what a warp does after a failed wait, all its lanes do)
    auto got = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait_abort(bar, parity & 1, abort) > 0);
    };

    if (warp >= 8 && warp < 16) {
        // ======================================================== codes to values
        const int which = warp >= 12, t = tid & 127;
        const uint8_t* const codes = which ? a.vc : a.kc;
        const uint32_t* const scales = which ? a.vs : a.ks;
        uint64_t* const full = which ? bs.v_full : bs.k_full;
        uint64_t* const empty = which ? bs.v_empty : bs.k_empty;
        uint64_t* const info = which ? bs.v_info : bs.k_info;
        unsigned char* const ring = sm + (which ? kOffV : kOffK);
        bool bad = false;
        while (ok && next_segment<kRT, true>(a, first, ch, cta, &u, u1, &s)) {
            auto block_of = [&](int tile) -> int {
                const int tok = tile * kTile + t;
                // (what no row sees may have been given up)
                if (tok > s.p_hi || (a.window && tok <= s.p_lo - a.window)) return -1;
                const int id = __ldg(a.table + (size_t)s.b * a.max_blocks + (tok >> a.bs_log2));
                if (id >= 0 && id < a.n_blocks) return id;
                bad = true;
                return -1;
            };
            uint4 next[4] = {};
            uint32_t sm_next = 0;
            auto load = [&](int tile, int id) {
                const int at = (tile * kTile + t) & ((1 << a.bs_log2) - 1);
                const size_t tok = (size_t)s.h << a.bs_log2 | at;
                const uint4* p = reinterpret_cast<const uint4*>(codes + (size_t)max(id, 0) * a.block_stride + tok * (kD / 2));
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = id >= 0 ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
                sm_next = id >= 0 ? __ldg(scales + ((size_t)id * a.kv_heads << a.bs_log2) + tok) : 0;
            };
            int id = s.n > 0 ? block_of(s.t0) : -1, id1 = s.n > 1 ? block_of(s.t0 + 1) : -1;
            if (s.n > 0) load(s.t0, id);
            for (int j = 0; ok && j < s.n; ++j) {
                const uint32_t g = G + j;
                const uint4 w[4] = {next[0], next[1], next[2], next[3]};
                const float sv = bf_lo(sm_next), mv = bf_hi(sm_next);
                const bool there = id >= 0;
                id = id1;
                if (j + 1 < s.n) load(s.t0 + j + 1, id);
                id1 = j + 2 < s.n ? block_of(s.t0 + j + 2) : -1;
                // the tile's largest magnitude
                const uint32_t mag = __float_as_uint(fmaxf(fabsf(mv), fabsf(fmaf(15.f, sv, mv))));
                const uint32_t top = __reduce_max_sync(0xffffffffu, mag);
                if (lane == 0) bs.most[which][g & 1][warp & 3] = top;
                const uint32_t on = __ballot_sync(0xffffffffu, there);
                warp_arrive(&bs.max_in[which], lane);
                ok = got(&bs.max_in[which], g);
                if (!ok) break;
                const uint32_t* most = bs.most[which][g & 1];
                const uint32_t all = max(max(most[0], most[1]), max(most[2], most[3]));
                const int e = min(max((int)(all >> 23) - 127, -100), 100);
                // (tile g - 4's exponent has been read: its products are done, or stage g & 1 would not come free)
                ok = g < 2 || got(&empty[g & 1], (g >> 1) + 1);
                if (!ok) break;
                if (lane == 0) {
                    if (which) bs.v_exp[g % kInfo] = e;
                    else {
                        bs.k_factor[g % kInfo] = pow2(e - kTop);
                        bs.there[g % kInfo][warp & 3] = on;
                    }
                }
                warp_arrive(&info[g % kInfo], lane);
                const float f = pow2(kTop - e);
                const __half2 s2 = __float2half2_rn(sv * f), s16 = __float2half2_rn(sv * f * 0.0625f), m2 = __float2half2_rn(mv * f);
                unsigned char* const to = ring + (g & 1) * kTileBytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(to + (i >> 1) * kHalf + sw128(t, (i & 1) * 4 + k)) = values8(x[k], s2, s16, m2);
                }
                fence_async_smem();
                warp_arrive(&full[g & 1], lane);
            }
            G += s.n;
        }
        if (bad) atomicOr(a.err, kErrBounds);
    } else if (warp == 16) {
        // ======================================================== MMA issue
        constexpr uint32_t id_qk = idesc_f32acc(0, 0, 0, 128, kTile);     // fp16, both K-major
        constexpr uint32_t id_pv = idesc_f32acc(0, 0, 1, 128, kD);        // V with its dims contiguous
        const uint32_t q0 = smem_u32(sm), k0 = smem_u32(sm + kOffK), v0 = smem_u32(sm + kOffV);
        uint32_t steps[2] = {0, 0}, segs = 0;                  // weights taken of each lane, segments with tiles
        while (ok && next_segment<kRT, true>(a, first, ch, cta, &u, u1, &s)) {
            if (s.n == 0) continue;
            const bool both = s.nr > 128;                      // both lanes take every tile
            const int n[2] = {both ? s.n : (s.n + 1) / 2, both ? s.n : s.n / 2};
            auto tile = [&](int i, int j) { return G + (both ? j : 2 * j + i); };
            auto qk = [&](int i, int j) -> bool {
                const uint32_t g = tile(i, j), st = g & 1;
                if (!got(&bs.k_full[st], g >> 1)) return false;
                tc_fence_after();
                const uint32_t qa = q0 + (both ? i : 0) * kTileBytes, kb = k0 + st * kTileBytes;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        mma_f16kind(tmem + i * 128, desc_sw128(qa + off, 16, 1024), desc_sw128(kb + off, 16, 1024), id_qk, kk > 0);
                    }
                    if (!both || i == 1) mma_commit(&bs.k_empty[st]);
                    mma_commit(&bs.s_full[i]);
                }
                __syncwarp();
                return true;
            };
            auto pv = [&](int i, int j) -> bool {
                const uint32_t g = tile(i, j), st = g & 1;
                if (!got(&bs.v_full[st], g >> 1) || !got(&bs.p_full[i], steps[i])) return false;
                ++steps[i];
                tc_fence_after();
                const uint32_t vb = v0 + st * kTileBytes;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + 256 + i * 128, tmem + i * 128 + kk * 8, desc_sw128(vb + kk * 2048, kHalf, 1024), id_pv,
                               j > 0 || kk > 0);
                    if (!both || i == 1) mma_commit(&bs.v_empty[st]);
                }
                __syncwarp();
                return true;
            };
            ok = got(&bs.q_full, segs);
            ++segs;
            for (int i = 0; i < 2; ++i)
                if (ok && n[i] > 0) ok = qk(i, 0);
            for (int j = 0; ok && j < n[0]; ++j)
                for (int i = 0; i < 2; ++i) {
                    if (ok && j < n[i]) ok = pv(i, j);
                    if (ok && j + 1 < n[i]) ok = qk(i, j + 1);
                }
            if (ok && elect_one()) mma_commit(&bs.o_full);
            __syncwarp();
            G += s.n;
        }
        // every MMA issued completes before TMEM is freed
        if (elect_one()) mma_commit(&bs.drain);
        __syncwarp();
        if (!mbar_wait(&bs.drain, 0)) ok = false;
    } else {
        // ======================================================== softmax: a thread a row
        const int i = warp >> 2, t = tid & 127;                // lane of the CTA, row in it
        const uint32_t base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t my_s = tmem + base + i * 128, my_o = tmem + base + 256 + i * 128;
        uint32_t steps = 0, segs = 0, meets = 0;
        // all softmax threads; false after a failed wait
        auto meet = [&]() {
            uint64_t* bar = &bs.met[meets & 1];
            warp_arrive(bar, lane);
            return got(bar, meets++ >> 1);
        };
        while (ok && next_segment<kRT, true>(a, first, ch, cta, &u, u1, &s)) {
            const bool both = s.nr > 128;
            const int row = both ? i * 128 + t : t;            // in the row tile
            const int tok = (s.row0 + row) / a.group;          // of the request's new tokens
            const bool on = row < s.nr;
            const size_t head = (size_t)(s.h * a.group + s.row0 + row - tok * a.group) * kD;
            const int p0 = s.len - s.nq, pos = on ? p0 + tok : -1;
            float factor = 0.f;                                // of this row's scores
            if (s.n > 0) {
                const uint4* x = reinterpret_cast<const uint4*>(a.q + (size_t)(s.q0 + (on ? tok : 0)) * a.q_row + (on ? head : 0));
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint4 v = on ? __ldg(x + k) : make_uint4(0, 0, 0, 0);
                    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                             __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                }
                m = max(m & 0xffffu, m >> 16);
                const int e = min(max((int)(m >> 7) - 127 - kTop, -120), 120);
                // a row that is not finite has no result: NaN
                factor = m >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(e) * fabsf(a.scale_log2);
                if (both || i == 0) {
                    const float inv = a.scale_log2 < 0.f ? -pow2(-e) : pow2(-e);
#pragma unroll 4
                    for (int k = 0; k < 16; ++k) {
                        const uint4 v = on ? __ldg(x + k) : make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(sm + i * kTileBytes + (k >> 3) * kHalf + sw128(t, k & 7)) =
                            make_uint4(half2_bits(bf_lo(v.x) * inv, bf_lo(v.z) * inv), half2_bits(bf_hi(v.x) * inv, bf_hi(v.z) * inv),
                                       half2_bits(bf_lo(v.y) * inv, bf_lo(v.w) * inv), half2_bits(bf_hi(v.y) * inv, bf_hi(v.w) * inv));
                    }
                }
                fence_async_smem();
                warp_arrive(&bs.q_full, lane);
            }
            const int lane_lo = p0 + (s.row0 + (both ? i * 128 : 0)) / a.group, lane_hi = s.p_hi;
            const int win = a.window ? a.window : 1 << 30;
            float ref = kLow, l = 0.f;
            const int n = both ? s.n : (s.n + 1 - i) / 2;
            for (int j = 0; j < n; ++j) {
                const int tile = both ? j : 2 * j + i;
                const uint32_t g = G + tile;
                const int t0 = (s.t0 + tile) * kTile;
                ok = got(&bs.s_full[i], steps) && got(&bs.k_info[g % kInfo], g / kInfo) && got(&bs.v_info[g % kInfo], g / kInfo);
                if (!ok) break;
                ++steps;
                tc_fence_after();
                const float sc = factor * bs.k_factor[g % kInfo];
                const int ve = bs.v_exp[g % kInfo];
                const uint4 there = *reinterpret_cast<const uint4*>(bs.there[g % kInfo]);
                const bool edge = t0 + kTile - 1 > lane_lo || t0 <= lane_hi - win ||
                                  (there.x & there.y & there.z & there.w) != 0xffffffffu;
                // this row's tokens of each 32, a bit each
                auto seen = [&](int c) -> uint32_t {
                    const int lo = pos - win + 1 - t0 - c * 32, hi = pos - t0 - c * 32;      // the first and the last
                    const uint32_t w = c == 0 ? there.x : c == 1 ? there.y : c == 2 ? there.z : there.w;
                    if (hi < 0 || lo > 31) return 0;
                    return w & (0xffffffffu >> (31 - min(hi, 31))) & (0xffffffffu << max(lo, 0));
                };
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    tmem_ld<32>(my_s + c * 32, x);
                    tmem_ld_wait();
                    tmem_regs_ready_n<32>(x);
                    if (edge) {
                        const uint32_t w = seen(c);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(w >> k & 1)) x[k] = -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 2) top = max3(top, x[k], x[k + 1]);
                }
                const float most = top == -INFINITY ? top : fmaf(top, sc, (float)ve);
                float fac = 1.f;
                if (most - ref > kRoom) {
                    const float now = most - kHead;
                    fac = ex2(ref - now);
                    ref = now;
                    l *= fac;
                }
                if (j > 0 && __any_sync(0xffffffffu, fac != 1.f)) {
                    // (the products before this tile's scores are complete)
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        float o[16];
                        tmem_ld<16>(my_o + c * 16, o);
                        tmem_ld_wait();
                        tmem_regs_ready_n<16>(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] *= fac;
                        tmem_st<16>(my_o + c * 16, o);
                    }
                }
                const float add = (float)ve - ref;
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[32], p[16];
                    tmem_ld<32>(my_s + c * 32, x);
                    tmem_ld_wait();
                    tmem_regs_ready_n<32>(x);
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = ex2(fmaf(x[k], sc, add));
                    if (edge) {
                        const uint32_t w = seen(c);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(w >> k & 1)) x[k] = 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        sum0 += x[k];
                        sum1 += x[k + 1];
                        p[k / 2] = __uint_as_float(half2_bits(x[k], x[k + 1]));
                    }
                    tmem_st<16>(my_s + c * 16, p);             // over scores that have been read
                }
                l = fmaf(sum0 + sum1, pow2(-ve), l);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&bs.p_full[i], lane);
            }
            if (!ok) break;
            G += s.n;
            // ---------------------------------------------------- out
            float f0 = 1.f, f1 = 0.f, m = ref, sum = l;        // factors of the two lanes' outputs
            if (s.n > 0) {
                ok = got(&bs.o_full, segs);
                ++segs;
                if (!ok) break;
                tc_fence_after();
                if (!both) {
                    bs.stat[i][t] = make_float2(ref, l);
                    ok = meet();
                    if (!ok) break;
                    const float2 x = bs.stat[0][t], y = bs.stat[1][t];
                    m = fmaxf(x.y != 0.f ? x.x : kLow, y.y != 0.f ? y.x : kLow);
                    f0 = x.y != 0.f ? ex2(x.x - m) : 0.f;
                    f1 = y.y != 0.f ? ex2(y.x - m) : 0.f;
                    sum = f0 * x.y + f1 * y.y;
                }
            }
            const float inv = sum == 0.f ? 0.f : s.parts == 1 ? pow2(-kTop) / sum : pow2(-kTop);
            const size_t slot = slot_of(s.v0, s.part);
            uint16_t* const out = a.out + (size_t)(s.q0 + tok) * a.out_row + head;
            float* const part = a.part_o + (slot * kRT + row) * kD;
            // a lane's own columns of its rows, or half of them of the rows that both have
            const int c0 = both ? 0 : i * 8, c1 = both ? 16 : c0 + 8;
#pragma unroll 1
            for (int c = c0; c < c1; c += 2) {
                float o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = 0.f;
                if (s.n > 0) {
                    tmem_ld<16>(both ? my_o + c * 8 : tmem + base + 256 + c * 8, o);
                    tmem_ld_wait();
                    tmem_regs_ready_n<16>(o);
                    if (!both) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = f0 == 0.f ? 0.f : o[k] * f0;
                        if (s.n > 1) {
                            float o1[16];
                            tmem_ld<16>(tmem + base + 384 + c * 8, o1);
                            tmem_ld_wait();
                            tmem_regs_ready_n<16>(o1);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (f1 != 0.f) o[k] = fmaf(o1[k], f1, o[k]);
                        }
                    }
                }
                if (!on) continue;
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = inv == 0.f ? 0.f : o[k] * inv;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // columns hold dims 0, 4, 1, 5, 2, 6, 3, 7 of each 8
                    const float* v = o + 8 * k;
                    const int d = (c + k) * 8;
                    if (s.parts == 1) {
                        *reinterpret_cast<uint4*>(out + d) = make_uint4(bf2(v[0], v[2]), bf2(v[4], v[6]), bf2(v[1], v[3]), bf2(v[5], v[7]));
                    } else {
                        *reinterpret_cast<float4*>(part + d) = make_float4(v[0], v[2], v[4], v[6]);
                        *reinterpret_cast<float4*>(part + d + 4) = make_float4(v[1], v[3], v[5], v[7]);
                    }
                }
            }
            tc_fence_before();
            if (s.parts > 1) {
                if (on && (both || i == 0)) reinterpret_cast<float2*>(a.part_ml)[slot * kRT + row] = make_float2(m, sum);
                ok = finish<kRT, kD>(a, s, tid, 256, &bs.last, meet);
                if (!ok) break;
            }
        }
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    const bool failed = __syncthreads_or(!ok);
    if (failed && tid == 0) atomicOr(a.err, kErrTimeout);
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

int smem_bytes(int n_req) { return kOffBars + (int)sizeof(Bars) + n_req * (int)sizeof(int) + 1024; }

}  // namespace

void chunk4_scratch(int sm_count, size_t* o_floats, size_t* ml_floats) {
    *o_floats = (size_t)sm_count * 2 * kRT * kD;
    *ml_floats = (size_t)sm_count * 4 * kRT;
}

cudaError_t set_chunk4_attrs() {
    return cudaFuncSetAttribute(chunk4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxBatch));
}

cudaError_t launch_chunk4(int sm_count, Args a, cudaStream_t st) {
    a.arrived_n = sm_count;
    chunk4_kernel<<<sm_count, kThreads, smem_bytes(a.n_req), st>>>(a);
    return cudaGetLastError();
}

}  // namespace kv8
}  // namespace srh
