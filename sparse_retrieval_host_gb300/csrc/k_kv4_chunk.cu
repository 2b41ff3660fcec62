// Attention over the paged 4-bit cache (kv4_attend) for requests of many query rows per KV head
// (prompt chunks, drafts of wide groups) on the 5th-generation tensor cores.
//
// Rows are the M dimension of both products, S = Q K^T and O = P V. Codes become fp16 values in
// shared memory once per tile of 128 tokens and are used by up to 256 rows:
//   k = (m + n s) 2^(14 - e), e the exponent of the tile's largest magnitude,
// one rounding, 2^-11 of the value at most, plus 16 steps of 2^-39 of the tile's largest where s and m become subnormal;
// the power of two goes into the scores' factor, V's into the exponent u = score + e of the weights 2^(u - ref), which
// are rounded to fp16, and is taken out of the softmax's sums again. A thread holds a row, so maxima and sums
// need no exchange; a row's reference moves only when a weight would pass 2^15.5.
//
// A CTA runs two lanes of 128 rows, each with its own S and O in TMEM (P lies over S), so that one
// lane's exponentials run beside the other's products. Of a row tile of more than 128 rows the lanes
// take the two halves, tile by tile of the same tokens; of one of up to 128 rows they take the same
// rows and every other tile, and add up at the end. Of 256 dims a row tile has 128 rows and K and V one stage each: both
// lanes take every tile of the same rows, each with all scores and weights and half of V's dims, as O has 256 columns and
// TMEM room for them and two S only that way (the third of the products and half of the exponentials that are made
// twice cost as much as twice the rows of 128 dims would).
//
// Per 128 tokens x 256 rows: 2,048 cycles of MMA at the fp16 rate, 1,024 of exponentials (32 a cycle, measured),
// 2,048 of shared memory (QK reads both operands: 1,024; PV one: 512; expanding writes 512).
//
// Roles: warps 0-3 and 4-7 softmax of the two lanes, 8-11 expand K, 12-15 V (a thread a token, the
// next tile's codes in registers), 16 issues the MMAs, 17 finds the segments. All waits are on mbarriers and bounded.
//
// Measured: four prompts of up to 1,024 tokens on up to 8,192, 32 / 8 heads of 128: 326 us with the join, 0.38 of the fp16 rate;
// some 4,400 cycles a full tile. Of those a warp's 128 columns from TMEM cost about 300 each time (they are read twice, once
// for the maximum and once for the weights: 96 registers hold 32 columns; 56 bytes are spilled, 36 of 256 dims), the
// scores of a scheduler's two warps on their way to weights 1,580. The tensor pipe is busy for 33 % of the kernel's time, which is
// thus 6,100 cycles a tile: starts and ends of the three to four row tiles of a CTA, and the wait for the last CTA, are the rest. Scores
// in registers (152 of them, by setmaxnreg): 386 us. Of as many products with 16 / 4 heads of 256: 416 us (8 rows at a time by
// the kernel of few rows: 1,463).
#include "kv4_split.cuh"
#include "umma.cuh"

namespace srh {
namespace kv8 {
namespace {

using namespace umma;
using namespace split;

constexpr int kExpand = 8, kIssue = 16, kPlan = 17;   // first warp that expands; those that issue MMAs and find segments
constexpr int kThreads = (kPlan + 1) * 32;
constexpr int kHalf = 16384;             // 128 rows of 64 fp16 values
constexpr int kTileBytes = 2 * kHalf;
constexpr int kOffK = 2 * kTileBytes;    // behind Q of the two lanes
constexpr int kOffV = kOffK + 2 * kTileBytes;
constexpr int kOffBars = kOffV + 2 * kTileBytes;
// DB: head_dim / 128.
template <int DB_>
struct Form {
    static constexpr int DB = DB_, RT = 256 / DB, D = 128 * DB;
    static constexpr bool HALVES = DB == 1;
    static constexpr int SW = DB == 1 ? 8 : 4;                 // units (half tiles; tiles) that a row tile's start and end take the time of
    static constexpr int ST = 2 / DB;                          // stages of K and of V
    static constexpr int kStage = DB * kTileBytes;
};
constexpr int kSegs = 4;                 // segments found ahead of their use
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
    uint64_t seg_full[kSegs], seg_empty[kSegs];   // a segment is found; every other warp has done with it
    Segment seg[kSegs];                  // h < 0: no more
    long long warp_sums[33];
    uint32_t tmem_base;
    int abort;
    uint32_t most[2][2][4];              // [K, V][tile & 1][warp]: largest magnitude
    alignas(16) uint32_t there[kInfo][4];            // tokens that exist, a bit each
    float k_factor[kInfo];               // 2^(e - 14)
    int v_exp[kInfo];                    // e
    float2 stat[2][128];                 // reference and sum of each lane's rows
    float factor[2][128];                // of each lane's rows' scores
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
// The eight values of a word of codes, as pairs (i, i + 4). A code in the low bits of 1024, or four bits
// up in those of 64, is exact there, and n without the 1024 or the 64 (without the product by s as 16 n times s / 16, whose
// bits a small s loses).
__device__ __forceinline__ uint4 values8(uint32_t w, __half2 s, __half2 m) {
    const __half2 k = __float2half2_rn(1024.f), k16 = __float2half2_rn(64.f);
    const uint32_t x = w >> 8;
    uint4 r;
    r.x = bits(__hfma2(__hsub2(as_half2((w & 0x000f000fu) | 0x64006400u), k), s, m));
    r.y = bits(__hfma2(__hsub2(as_half2((w & 0x00f000f0u) | 0x54005400u), k16), s, m));
    r.z = bits(__hfma2(__hsub2(as_half2((x & 0x000f000fu) | 0x64006400u), k), s, m));
    r.w = bits(__hfma2(__hsub2(as_half2((x & 0x00f000f0u) | 0x54005400u), k16), s, m));
    return r;
}
__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float4 lds_float4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}

// Values of tokens whose bit is not set become `none`.
__device__ __forceinline__ void mask32(uint32_t seen, float (&x)[32], float none) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (!(seen >> k & 1)) x[k] = none;
}

template <int DB>
__global__ void __launch_bounds__(kThreads, 1) chunk4_kernel(const __grid_constant__ Args a) {
    using F = Form<DB>;
    constexpr int kRT = F::RT, kD = F::D, ST = F::ST;
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
            mbar_init(&bs.s_full[i], 1);
            mbar_init(&bs.p_full[i], 4);
            mbar_init(&bs.met[i], 8);
        }
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(&bs.k_info[i], 4);
            mbar_init(&bs.v_info[i], 4);
        }
        mbar_init(&bs.max_in[0], 4);
        mbar_init(&bs.max_in[1], 4);
        mbar_init(&bs.q_full, 8);
        mbar_init(&bs.o_full, 1);
        mbar_init(&bs.drain, 1);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&bs.seg_full[i], 1);
            mbar_init(&bs.seg_empty[i], kPlan);
        }
        bs.abort = 0;
        fence_mbar_init();
    }
    Chunks ch;
    if (!count<kRT, F::HALVES, F::SW, kThreads>(a, first, bs.warp_sums, &ch)) {            // every thread
        if (blockIdx.x == 0 && tid == 0) a.ctrl[1] = 0;
        return;
    }
    if (tid == 0) {
        a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);            // no row tile goes on from this chunk, so far
        if (blockIdx.x == 0) a.ctrl[1] = ch.n;
    }
    if (warp == kIssue) tmem_alloc(&bs.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bs.tmem_base;                        // S of the lanes at 0 and 128, O at 256 and 384
    const int cta = blockIdx.x;
    bool ok = true;
    uint32_t G = 0;                                            // tiles before this segment
    // (what a warp does after a failed wait, all its lanes do)
    auto got = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait_abort(bar, parity & 1, abort) > 0);
    };

    // segment k, once it is found; false: there are no more, or the wait failed
    auto take = [&](uint32_t k) {
        ok = got(&bs.seg_full[k % kSegs], k / kSegs);
        return ok && bs.seg[k % kSegs].h >= 0;
    };
    auto release = [&](uint32_t k) { warp_arrive(&bs.seg_empty[k % kSegs], lane); };

    if (warp == kPlan) {
        // ======================================================== segments, and their queries into L2
        int u = ch.begin(cta);
        const int u1 = ch.begin(cta + 1);
        bool more = true;
        for (uint32_t k = 0; ok && more; ++k) {
            Segment s;
            more = next_segment<kRT, F::HALVES, F::SW>(a, first, ch, cta, &u, u1, &s);
            if (!more) s.h = -1;
            ok = k < kSegs || got(&bs.seg_empty[k % kSegs], k / kSegs + 1);
            if (!ok) break;
            if (lane == 0) bs.seg[k % kSegs] = s;
            warp_arrive(&bs.seg_full[k % kSegs], lane);
            for (int r = lane; more && r < s.nr; r += 32) {
                const int tok = by_group(a, s.row0 + r);
                const uint16_t* x = a.q + (size_t)(s.q0 + tok) * a.q_row + (size_t)(s.h * a.group + s.row0 + r - tok * a.group) * kD;
#pragma unroll
                for (int d = 0; d < kD; d += 64) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(x + d));
            }
        }
    } else if (warp >= kExpand && warp < kIssue) {
        // ======================================================== codes to values
        const int which = warp >= kExpand + 4, t = tid & 127;          // K or V, token of the tile
        const uint8_t* const codes = which ? a.vc : a.kc;
        const uint32_t* const scales = which ? a.vs : a.ks;
        uint64_t* const full = which ? bs.v_full : bs.k_full;
        uint64_t* const empty = which ? bs.v_empty : bs.k_empty;
        uint64_t* const info = which ? bs.v_info : bs.k_info;
        const uint32_t ring = smem_u32(sm) + (which ? kOffV : kOffK);
        bool bad = false;
        for (uint32_t k = 0; ok && take(k); ++k) {
            const Segment& s = bs.seg[k % kSegs];
            const int n = s.n, first_tile = s.t0, p_hi = s.p_hi, head_tok = s.h << a.bs_log2;
            const int see_first = a.window ? s.p_lo - a.window + 1 : 0;
            const int32_t* const table = a.table + (size_t)s.b * a.max_blocks;
            auto block_of = [&](int tile) -> int {
                const int tok = tile * kTile + t;
                // (what no row sees may have been given up)
                if (tok > p_hi || tok < see_first) return -1;
                const int id = __ldg(table + (tok >> a.bs_log2));
                if (id >= 0 && id < a.n_blocks) return id;
                bad = true;
                return -1;
            };
            uint4 next[4] = {};
            uint32_t sm_next = 0;
            auto load = [&](int tile, int id, int part) {      // 128 dims
                const int tok = head_tok | ((tile * kTile + t) & ((1 << a.bs_log2) - 1));
                const uint4* p = reinterpret_cast<const uint4*>(codes + (size_t)max(id, 0) * a.block_stride + tok * (kD / 2) + part * 64);
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = id >= 0 ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
                if (part == 0) sm_next = id >= 0 ? __ldg(scales + ((size_t)id * a.kv_heads << a.bs_log2) + tok) : 0;
            };
            int id = n > 0 ? block_of(first_tile) : -1, id1 = n > 1 ? block_of(first_tile + 1) : -1;
            if (n > 0) load(first_tile, id, 0);
            for (int j = 0; ok && j < n; ++j) {
                const uint32_t g = G + j;
                uint4 w[4] = {next[0], next[1], next[2], next[3]};
                const float sv = bf_lo(sm_next), mv = bf_hi(sm_next);
                const bool there = id >= 0;
                if (DB == 2) load(first_tile + j, id, 1);
                id = id1;
                if (DB == 1 && j + 1 < n) load(first_tile + j + 1, id, 0);
                id1 = j + 2 < n ? block_of(first_tile + j + 2) : -1;
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
                // (V's as in the kernel of few rows: of all zeros weights would be 2^100 in the softmax's sum, too many for fp32)
                const int e = min(max((int)(all >> 23) - 127, which ? -64 : -100), 100);
                const float f = pow2(kTop - e);
                const __half2 s2 = __float2half2_rn(sv * f), m2 = __float2half2_rn(mv * f);
                auto publish = [&] {
                    if (lane == 0) {
                        if (which) bs.v_exp[g % kInfo] = e;
                        else {
                            bs.k_factor[g % kInfo] = pow2(e - kTop);
                            bs.there[g % kInfo][warp & 3] = on;
                        }
                    }
                    warp_arrive(&info[g % kInfo], lane);
                };
                // (tile g - 4's exponent has been read. Of one stage: tile g - 2's products are done, and those of a lane's
                // queries come after its weights of tile g - 3; it need not wait for the stage, which lane 1 has longest)
                if (ST == 1) publish();
                ok = g < ST || got(&empty[g % ST], g / ST + 1);
                if (!ok) break;
                // (of two: tile g - 4's products are done, or the stage would not come free)
                if (ST == 2) publish();
#pragma unroll 1
                for (int part = 0; part < DB; ++part) {
                    const uint32_t to = ring + (g % ST) * F::kStage + part * kTileBytes;
                    if (part == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = next[i];
                        if (j + 1 < n) load(first_tile + j + 1, id, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) sts128(to + (i >> 1) * kHalf + sw128(t, (i & 1) * 4 + k), values8(x[k], s2, m2));
                    }
                }
                fence_async_smem();
                warp_arrive(&full[g % ST], lane);
            }
            G += n;
            release(k);
        }
        if (bad) atomicOr(a.err, kErrBounds);
    } else if (warp == kIssue) {
        // ======================================================== MMA issue
        constexpr uint32_t id_qk = idesc_f32acc(0, 0, 0, 128, kTile);     // fp16, both K-major
        constexpr uint32_t id_pv = idesc_f32acc(0, 0, 1, 128, 128);       // V with its dims contiguous
        const uint32_t q0 = smem_u32(sm), k0 = smem_u32(sm + kOffK), v0 = smem_u32(sm + kOffV);
        uint32_t steps[2] = {0, 0}, segs = 0;                  // weights taken of each lane, segments with tiles
        for (uint32_t seg = 0; ok && take(seg); ++seg) {
            const Segment s = bs.seg[seg % kSegs];
            release(seg);
            if (s.n == 0) continue;
            const bool both = DB == 2 || s.nr > 128;           // both lanes take every tile
            const bool rows = DB == 1 && both;                 // .. of rows of their own
            const int n[2] = {both ? s.n : (s.n + 1) / 2, both ? s.n : s.n / 2};
            auto tile = [&](int i, int j) { return G + (both ? j : 2 * j + i); };
            auto qk = [&](int i, int j) -> bool {
                const uint32_t g = tile(i, j), st = g % ST;
                if (!got(&bs.k_full[st], g / ST)) return false;
                tc_fence_after();
                const uint32_t qa = q0 + (rows ? i : 0) * kTileBytes, kb = k0 + st * F::kStage;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8 * DB; ++kk) {
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
                const uint32_t g = tile(i, j), st = g % ST;
                if (!got(&bs.v_full[st], g / ST) || !got(&bs.p_full[i], steps[i])) return false;
                ++steps[i];
                tc_fence_after();
                const uint32_t vb = v0 + st * F::kStage + (DB == 2 ? i * kTileBytes : 0);
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
        for (uint32_t seg = 0; ok && take(seg); ++seg) {
            const Segment& s = bs.seg[seg % kSegs];
            const bool both = DB == 2 || s.nr > 128, rows = DB == 1 && both;
            const int row = rows ? i * 128 + t : t;            // in the row tile
            const int tok = by_group(a, s.row0 + row);          // of the request's new tokens
            const bool on = row < s.nr;
            const int head = (s.h * a.group + s.row0 + row - tok * a.group) * kD;
            const int p0 = s.len - s.nq, pos = on ? p0 + tok : -1;
            float factor = 0.f;                                // of this row's scores
            if (s.n > 0) {
                // the warp's 32 rows, two (of 256 dims one) at a time with 16 bytes a lane
                constexpr int kLanes = 16 * DB;
                const long long q_at = (long long)(s.q0 + tok) * a.q_row + head;
                uint4 v[16];
                const int piece = lane & (kLanes - 1), r0 = (rows ? i * 128 : 0) + (warp & 3) * 32;
#pragma unroll 1
                for (int y0 = 0; y0 < DB; ++y0) {
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const int from = DB == 1 ? 2 * y + (lane >> 4) : y0 * 16 + y;
                        const long long at = __shfl_sync(0xffffffffu, q_at, from);
                        v[y] = r0 + from < s.nr ? __ldg(reinterpret_cast<const uint4*>(a.q + at) + piece) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const int r = DB == 1 ? 2 * y + (lane >> 4) : y0 * 16 + y;     // of the warp's
                        uint32_t m = __vmaxu2(__vmaxu2(v[y].x & 0x7fff7fffu, v[y].y & 0x7fff7fffu),
                                              __vmaxu2(v[y].z & 0x7fff7fffu, v[y].w & 0x7fff7fffu));
#pragma unroll
                        for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
                        m = max(m & 0xffffu, m >> 16);
                        const int e = min(max((int)(m >> 7) - 127 - kTop, -120), 120);
                        // a row that is not finite has no result: NaN
                        if (piece == 0)
                            bs.factor[i][(warp & 3) * 32 + r] = m >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(e) * fabsf(a.scale_log2);
                        if (rows || i == 0) {
                            const float inv = a.scale_log2 < 0.f ? -pow2(-e) : pow2(-e);
                            sts128(smem_u32(sm) + i * kTileBytes + (piece >> 3) * kHalf + sw128((warp & 3) * 32 + r, piece & 7),
                                   make_uint4(half2_bits(bf_lo(v[y].x) * inv, bf_lo(v[y].z) * inv), half2_bits(bf_hi(v[y].x) * inv, bf_hi(v[y].z) * inv),
                                              half2_bits(bf_lo(v[y].y) * inv, bf_lo(v[y].w) * inv), half2_bits(bf_hi(v[y].y) * inv, bf_hi(v[y].w) * inv)));
                        }
                    }
                }
                fence_async_smem();
                warp_arrive(&bs.q_full, lane);
                factor = bs.factor[i][t];
            }
            const int lane_lo = p0 + by_group(a, s.row0 + (rows ? i * 128 : 0)), lane_hi = s.p_hi;
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
                // Loops that are not unrolled: four roles' code has to share the instruction caches.
                float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    tmem_ld<32>(my_s + c * 32, x);
                    tmem_ld_wait();
                    tmem_regs_ready_n<32>(x);
                    if (edge) mask32(seen(c), x, -INFINITY);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) tops[k >> 1 & 1] = max3(tops[k >> 1 & 1], x[k], x[k + 1]);
                }
                const float top = fmaxf(tops[0], tops[1]), most = top == -INFINITY ? top : fmaf(top, sc, (float)ve);
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
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        tmem_ld<32>(my_o + c * 32, o);
                        tmem_ld_wait();
                        tmem_regs_ready_n<32>(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= fac;
                        tmem_st<16>(my_o + c * 32, reinterpret_cast<const float(&)[16]>(o[0]));
                        tmem_st<16>(my_o + c * 32 + 16, reinterpret_cast<const float(&)[16]>(o[16]));
                    }
                }
                const u64 sc2 = pack(sc, sc), to2 = pack((float)ve - ref, (float)ve - ref);
                // Scores so large that ref's rounding counts are taken as above, rounded before the difference: the row's
                // largest would lose its weight else.
                const bool far = __any_sync(0xffffffffu, fabsf(ref) > 1e6f && ref != kLow);
                u64 sums[2] = {0, 0};
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float x[32], p[16];
                    tmem_ld<32>(my_s + c * 32, x);
                    tmem_ld_wait();
                    tmem_regs_ready_n<32>(x);
                    if (far) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = fmaf(x[k], sc, (float)ve) - ref;
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) unpack(fma2(pack(x[k], x[k + 1]), sc2, to2), x[k], x[k + 1]);
                    }
                    if (edge) mask32(seen(c), x, -INFINITY);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float e0 = ex2(x[k]), e1 = ex2(x[k + 1]);
                        sums[k >> 1 & 1] = add2(sums[k >> 1 & 1], pack(e0, e1));
                        p[k / 2] = __uint_as_float(half2_bits(e0, e1));
                    }
                    tmem_st<16>(my_s + c * 16, p);             // over scores that have been read
                }
                {
                    float s0, s1;
                    unpack(add2(sums[0], sums[1]), s0, s1);
                    l = fmaf(s0 + s1, pow2(-ve), l);
                }
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
            if (s.parts > 1) {
                if (on && (rows || i == 0)) reinterpret_cast<float2*>(a.part_ml)[slot * kRT + row] = make_float2(m, sum);
                if (tid == 0 && s.part == 0) a.meta[cta] = make_int4(s.parts | s.nr << 12, s.q0, s.row0, s.h);
            }
            // A lane's own columns of its rows, or half of them of the rows that both have: 64 at a time through the
            // warp's 8 KB of what held Q, so that rows go out in whole lines (a thread writing its own row: 6 us).
            const uint32_t own = smem_u32(sm) + warp * 8192;   // [32 rows][16 pieces], a row's turned by its number
            const long long out_at = (long long)(s.q0 + tok) * a.out_row + head;
            const int first_row = (rows ? i * 128 : 0) + (warp & 3) * 32;
#pragma unroll 1
            for (int half = both ? 0 : i; half < (both ? 2 : i + 1); ++half) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float o[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = 0.f;
                    if (s.n > 0) {
                        const uint32_t col = half * 64 + c * 16;
                        tmem_ld<16>((both ? my_o : tmem + base + 256) + col, o);
                        tmem_ld_wait();
                        tmem_regs_ready_n<16>(o);
                        if (!both) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = f0 == 0.f ? 0.f : o[k] * f0;
                            if (s.n > 1) {
                                float o1[16];
                                tmem_ld<16>(tmem + base + 384 + col, o1);
                                tmem_ld_wait();
                                tmem_regs_ready_n<16>(o1);
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (f1 != 0.f) o[k] = fmaf(o1[k], f1, o[k]);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = inv == 0.f ? 0.f : o[k] * inv;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // columns hold dims 0, 4, 1, 5, 2, 6, 3, 7 of each 8
                        const float* v = o + 8 * k;
                        const int piece = c * 4 + 2 * k;
                        sts128(own + lane * 256 + ((piece ^ (lane & 15)) << 4),
                               make_uint4(__float_as_uint(v[0]), __float_as_uint(v[2]), __float_as_uint(v[4]), __float_as_uint(v[6])));
                        sts128(own + lane * 256 + ((piece + 1 ^ (lane & 15)) << 4),
                               make_uint4(__float_as_uint(v[1]), __float_as_uint(v[3]), __float_as_uint(v[5]), __float_as_uint(v[7])));
                    }
                }
                __syncwarp();
#pragma unroll 4
                for (int y = 0; y < 32; y += 2) {
                    const int r = y + (lane >> 4), c4 = lane & 15, to = first_row + r;
                    const float4 v = lds_float4(own + r * 256 + ((c4 ^ (r & 15)) << 4));
                    const long long at = __shfl_sync(0xffffffffu, out_at, r);
                    if (to >= s.nr) continue;
                    const int d = (DB == 2 ? i * 128 : 0) + half * 64 + c4 * 4;
                    if (s.parts == 1) {
                        *reinterpret_cast<uint2*>(a.out + at + d) = make_uint2(bf2(v.x, v.y), bf2(v.z, v.w));
                    } else {
                        *reinterpret_cast<float4*>(a.part_o + (slot * kRT + to) * kD + d) = v;
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            release(seg);
            ok = meet();                                       // Q's place is free for the next queries
        }
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    const bool failed = __syncthreads_or(!ok);
    if (failed && tid == 0) atomicOr(a.err, kErrTimeout);
    if (warp == kIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of split row tiles together, in chunk order: part i has reference m_i, sum l_i and outputs O_i of each
// row, out = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i. A job is 32 rows, a warp and a 16-byte piece per lane
// each, four rows under way; of many parts (one long request) 4 rows, whose parts the warps share. (The last
// CTA to write its part joining them took 40 to 80 us for 256 rows, by itself.)
constexpr int kJoinThreads = 256, kFewParts = 12, kMostChunks = 512;
template <int DB>
__global__ void __launch_bounds__(kJoinThreads) join4_kernel(const __grid_constant__ Args a) {
    constexpr int kRT = Form<DB>::RT, kD = Form<DB>::D;
    __shared__ long long warp_sums[33];
    __shared__ int4 item[kMostChunks];
    __shared__ int jobs_before[kMostChunks], begins[kMostChunks];
    __shared__ float4 acc_s[8][4][32];
    __shared__ float sum_s[8][4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    const int n = min(a.ctrl[1], kMostChunks);
    int n_items = 0, n_jobs = 0;
    for (int base = 0; base < n; base += kJoinThreads) {
        const int v = base + tid;
        int4 it = v < n ? __ldcg(&a.meta[v]) : make_int4(0, 0, 0, 0);
        int parts = it.x & 0xfff;
        const int nr = it.x >> 12;
        if (parts > n - v || nr > kRT) parts = 0;              // (a call that gave up)
        const int jobs = DB * (parts == 0 ? 0 : parts <= kFewParts ? (nr + 31) / 32 : (nr + 3) / 4);
        long long total;
        const long long incl = block_scan(jobs ? (1ll << 32) + jobs : 0, warp_sums, &total);
        if (jobs) {
            const int k = n_items + (int)(incl >> 32) - 1;
            item[k] = it;
            begins[k] = v;
            jobs_before[k] = n_jobs + (int)(incl & 0xffffffff) - jobs;
        }
        n_items += (int)(total >> 32);
        n_jobs += (int)(total & 0xffffffff);
    }
    __syncthreads();
    const float2* const ml = reinterpret_cast<const float2*>(a.part_ml);
    for (int job = blockIdx.x; job < n_jobs; job += gridDim.x) {
        const int k = last_not_above(jobs_before, n_items, job);
        const int4 it = item[k];
        const int parts = it.x & 0xfff, nr = it.x >> 12, v0 = begins[k], j = job - jobs_before[k], at = j / DB;
        const int d0 = DB == 2 ? (j & 1) * 128 : 0;            // of the 128 dims of this job
        const bool few = parts <= kFewParts;
        // four rows of this warp's, and its parts of them
        const int r0 = few ? at * 32 + warp * 4 : at * 4;
        const int i0 = few ? 0 : parts * warp / 8, i1 = few ? parts : parts * (warp + 1) / 8;
        float m[4], sum[4];
        float4 acc[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            // the row's largest reference, of all its parts: a lane each
            m[y] = kLow;
            for (int i = lane; i < parts && r0 + y < nr; i += 32) {
                const float2 st = __ldcg(&ml[slot_of(v0, i) * kRT + r0 + y]);
                if (st.y != 0.f) m[y] = fmaxf(m[y], st.x);
            }
            sum[y] = 0.f;
            acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m[y] = fmaxf(m[y], __shfl_xor_sync(0xffffffffu, m[y], o));
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const size_t row = slot_of(v0, i) * kRT + min(r0 + y, nr - 1);
                const float2 st = __ldcg(&ml[row]);
                const float4 o = __ldcg(reinterpret_cast<const float4*>(a.part_o + row * kD + d0) + lane);
                const float f = st.y != 0.f ? ex2(st.x - m[y]) : 0.f;
                sum[y] = fmaf(f, st.y, sum[y]);
                // (a part with no weight does not count, whatever it holds)
                acc[y].x = f != 0.f ? fmaf(f, o.x, acc[y].x) : acc[y].x;
                acc[y].y = f != 0.f ? fmaf(f, o.y, acc[y].y) : acc[y].y;
                acc[y].z = f != 0.f ? fmaf(f, o.z, acc[y].z) : acc[y].z;
                acc[y].w = f != 0.f ? fmaf(f, o.w, acc[y].w) : acc[y].w;
            }
        }
        if (!few) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                acc_s[warp][y][lane] = acc[y];
                if (lane == 0) sum_s[warp][y] = sum[y];
            }
            __syncthreads();
            if (warp < 4) {
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float4 o = acc_s[w][warp][lane];
                    t.x += o.x;
                    t.y += o.y;
                    t.z += o.z;
                    t.w += o.w;
                    l += sum_s[w][warp];
                }
                acc[0] = t;
                sum[0] = l;
            }
            __syncthreads();
            if (warp >= 4) continue;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (!few && y > 0) break;
            const int row = few ? r0 + y : r0 + warp;
            if (row >= nr) continue;
            const float inv = sum[y] == 0.f ? 0.f : 1.f / sum[y];
            const int rr = it.z + row, tok = by_group(a, rr);
            *reinterpret_cast<uint2*>(a.out + (size_t)(it.y + tok) * a.out_row + (size_t)(it.w * a.group + rr - tok * a.group) * kD +
                                      d0 + lane * 4) =
                make_uint2(bf2(acc[y].x * inv, acc[y].y * inv), bf2(acc[y].z * inv, acc[y].w * inv));
        }
    }
}

int smem_bytes(int n_req) { return kOffBars + (int)sizeof(Bars) + n_req * (int)sizeof(int) + 1024; }

}  // namespace

void chunk4_scratch(int sm_count, size_t* o_floats, size_t* ml_floats, size_t* meta) {
    static_assert(Form<1>::RT * Form<1>::D == Form<2>::RT * Form<2>::D, "parts of one size");
    *o_floats = (size_t)sm_count * 2 * Form<1>::RT * Form<1>::D;
    *ml_floats = (size_t)sm_count * 4 * Form<1>::RT;
    *meta = (size_t)sm_count;            // a chunk per CTA
}

cudaError_t set_chunk4_attrs() {
    cudaError_t e = cudaFuncSetAttribute(chunk4_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxBatch));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(chunk4_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxBatch));
    return e;
}

cudaError_t launch_chunk4(int sm_count, int head_dim, const Args& a, cudaStream_t st) {
    if (sm_count > kMostChunks) return cudaErrorInvalidValue;
    if (head_dim == 128) chunk4_kernel<1><<<sm_count, kThreads, smem_bytes(a.n_req), st>>>(a);
    else chunk4_kernel<2><<<sm_count, kThreads, smem_bytes(a.n_req), st>>>(a);
    return cudaGetLastError();
}
cudaError_t launch_join4(int sm_count, int head_dim, const Args& a, cudaStream_t st) {
    return launch_k(head_dim == 128 ? join4_kernel<1> : join4_kernel<2>, dim3((unsigned)(4 * sm_count)), dim3(kJoinThreads), 0, st,
                    true, a);
}

}  // namespace kv8
}  // namespace srh
