// Attention over the paged 8-bit cache (kv8_attend), on the 5th-generation
// tensor cores straight from the e4m3 codes.
//
//   o_r = sum_t w_rt V_t / sum_t w_rt,  w_rt = exp(scale <q_r, K_t>),
//   K_t = kc_t * ks(block of t), V_t = vc_t * vs(block of t)
//
// Tokens are the M dimension of both products, so a cache row never leaves the
// form it is stored in:
//   S^T[t, r]  = kc[t, :] . q[r, :]      A = code tile (K-major), B = queries
//   O^T[d, r] += vc[:, d] . p[:, r]      A = the same kind of tile read MN-major
// kind::f8f6f4 takes 8-bit operands on both sides. A query row is scaled by a
// power of two to a largest magnitude in [128, 256) and split into two e4m3
// terms, hi = e4m3(q), lo = e4m3(q - hi): 4 + 4 significant bits, which is bf16
// exactly. The two terms are two columns of one MMA (N = 2 * rows), so a tile is
// read from shared memory once for both; having columns of its own, the second
// term is held 16 times larger, which takes e4m3's smallest steps 16 times
// further down.
//
// Block scales: ks multiplies the score, one factor per thread (thread = TMEM
// lane = token). vs goes into the exponent: u = s + log2(vs), p = 2^(u - ref), so
// the column p holds what the token contributes, and the rounding of p is
// relative to the largest contribution; the softmax sum takes p / vs in fp32.
//
// Weights are rounded to fp16 and split into three e5m2 terms, p = hi + mid + lo:
// within 2^-9 (half of bf16's step), or half of e5m2's smallest step, 2^-17. The
// running reference of a row is set so that its maximum's weight is 2^10, and is moved
// only when a weight would pass 2^15.75 (e5m2 ends at 57,344): what a small weight may
// lose is 2^-27 of the row's largest contribution, so that 131,072 tokens behind one
// that takes nearly all lose 2^-10 of it together at the very most. (Two e4m3 terms
// reach 2^-15 only, below which the long tail of a row with one large weight came out
// as nothing: 8,192 tokens with a tenth of the weight between them lost all of it.)
// One vote of the softmax threads per tile says whether a reference moves; the
// maximum itself, the rescaling of the sums and of O^T in TMEM only happen then (the
// first tile, then the more rarely the more tokens a row has seen).
//
// Work: a "row tile" is RT of the (token, head) rows that share a KV head of a
// request; its tokens are cut into tiles of 128. Every (request, KV head, row
// tile, token tile) is a unit. The U units, counted from the lengths on the
// device, are cut into chunks of equal numbers, one per CTA. Of many units 12/16
// are cut so, 3/16 and 1/16 into as many smaller chunks that CTAs take as they come
// free (SMs run at different speeds: with one chunk each, the last CTA of a
// bandwidth-bound batch ended 8 % after the average). So ragged batches and single
// long requests both fill the SMs, and nothing depends on host knowledge of lengths. An item whose units fall into several chunks leaves
// fp32 partial sums, which a second kernel joins in chunk order: who ran a
// chunk does not show, and results repeat bit for bit.
//
// Roles: 4 to 16 softmax warps (a thread holds one token and 16 rows; they also
// bring queries in and outputs out), one TMA warp (one box per block of tokens
// and 128 values, into a ring of 16 KB slots), one MMA warp. QK of tile j + 1 is
// issued before PV of tile j. Every wait is bounded; on a timeout the CTA records
// it, lets its copies and MMAs end, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv8_internal.cuh"
#include "umma.cuh"

namespace srh {
namespace kv8 {
namespace {

using namespace umma;

constexpr int kTile = 128;               // tokens per tile
constexpr int kSlotBytes = kTile * 128;  // 128 tokens x 128 dims
constexpr float kLow = -1e30f;           // reference of a row that has seen no token
constexpr float kHead = 10.f;            // log2 of the weight that a new reference gives a row's maximum
constexpr float kRoom = 15.75f;          // a row's reference moves when a weight would pass 2^15.75 = 55,109
constexpr float kLoScale = 16.f;         // factor of a query's second term

// Rounds of chunks and where they begin, in sixteenths of the units.
constexpr int kRounds = 3;
constexpr int kRoundsFrom = 192;   // units per CTA
__device__ __forceinline__ int cut(int r) { return r == 0 ? 0 : r == 1 ? 12 : r == 2 ? 15 : 16; }

// DB: head_dim / 128. RT: rows per row tile. SHARED: V = K.
template <int DB_, int RT_, bool SHARED_>
struct Shape {
    static constexpr int DB = DB_, RT = RT_;
    static constexpr bool SHARED = SHARED_;
    static constexpr int N = 2 * RT;                       // hi and lo columns
    // The three terms of the weights are columns of one PV product where TMEM has room
    // for O^T's three parts (a fourth of zeros fills 16-row tiles up to whole 32-byte
    // rows). Else (64 rows of 512 dims) hi and mid are for the first TWO times 128 dims,
    // as far as the room goes, and terms follow each other into the same columns
    // otherwise (32 requests of 32,768 latent rows: 162 us; with TWO = 0 169).
    static constexpr bool CAT = 3 * DB * RT + N <= 512;
    static constexpr int ON = !CAT ? RT : RT == 16 ? 64 : 3 * RT;   // O^T columns per 128 dims
    static constexpr int TWO = CAT ? 0 : 2;
    // O^T's first column of 128 dims: hi, then mid and lo RT columns further on each, where apart
    static __host__ __device__ constexpr int o_at(int mb) { return CAT ? mb * ON : (mb + (mb < TWO ? mb : TWO)) * RT; }
    static constexpr int COLS = N + DB * ON + TWO * RT;
    static constexpr int ALLOC = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static constexpr int kQBytes = DB * N * 128;
    static constexpr int kPitch = RT == 64 ? 64 : 32;      // bytes of one token's row of a part of p
    static constexpr int kPart = kTile * kPitch;           // parts: a term each, or two of 16-row tiles
    static constexpr int kPBytes = (RT == 16 ? 2 : 3) * kPart;
    // byte offset of 16-byte piece c of token t's weights, pieces of hi first, then mid, lo
    static __device__ __forceinline__ uint32_t p_at(uint32_t t, uint32_t c) {
        constexpr uint32_t per = kPitch / 16;
        const uint32_t x = kPitch == 64 ? ((t >> 1) & 3u) : ((t >> 2) & 1u);
        return (c / per) * kPart + t * kPitch + ((c % per ^ x) << 4);
    }
    // CTAs per SM: four hide more of a decode step's latencies than fewer with longer
    // rings do (64 requests of up to 16,384 tokens: 204 us; three 208, two 229)
    static constexpr int CTAS = DB == 1 ? (RT == 16 ? 4 : 2) : DB == 2 && RT == 16 ? 2 : 1;
    // rounds of chunks, where a CTA's switches between segments overlap other CTAs' tiles
    // (alone on its SM a CTA is better off with one chunk: 256 requests of up to 32,768
    // latent rows 629 us, 677 in rounds; prompts of 512 tokens of 256-dim heads 715 and 739)
    static constexpr int ROUNDS = CTAS > 1 ? kRounds : 1;
    // 16 KB slots of the ring (128 tokens x 128 dims); K tile j + 1 is taken before V
    // tile j is given back, so two tiles must fit
    static constexpr int SLOTS = DB == 1 ? (RT == 16 ? 2 : 5) : DB == 2 ? (RT == 16 ? 5 : 9) : RT == 16 ? 12 : RT == 32 ? 10 : 8;
    static_assert(SLOTS >= 2 * DB && SLOTS / DB + 2 < 8, "two tiles must fit the ring, and fewer than the scales held");
    // softmax: a thread holds CT columns of one token, CG groups of 4 warps share the
    // columns. (32 columns a thread, for 64-row tiles with two CTAs per SM, need more
    // than the 96 registers there are: a prompt chunk of 128-dim heads took 613 us
    // with them and took 545 with tiles of 32 rows at the time, now 593.)
    static constexpr int CT = 16;
    static constexpr int CG = RT / CT;
    static constexpr int SOFT = 128 * CG;                  // softmax threads
    static constexpr int THREADS = SOFT + 64;
    // A segment's start and end take about as long as so many tiles, and are counted
    // as such (4 against none: 16 requests of up to 5 drafted tokens 50 -> 47 us, the
    // latent batch 168 -> 162; with four CTAs per SM they overlap others' tiles: 1
    // against 4 in the decode batch, 204 against 205 us).
    static constexpr int SWITCH = DB == 1 && RT == 16 ? 1 : 4;
    static constexpr int kOffQ = SLOTS * kSlotBytes;
    static constexpr int kOffP = kOffQ + kQBytes;
    static constexpr int kOffBars = kOffP + kPBytes;
};

struct Args {
    const uint16_t* q;
    uint16_t* out;
    long long q_row, out_row;
    const int32_t* cu;
    const int32_t* len;
    const int32_t* table;
    const float* ks;
    const float* vs;
    float* part_o;
    float* part_ml;
    int4* meta;
    int* ctrl;                                   // [0] chunks handed out, [1] chunks of this call
    uint32_t* err;
    int n_req, n_rows, kv_heads, group;          // group = query heads / kv_heads
    int bs_log2, n_blocks, max_blocks;
    float scale_log2;
    unsigned long long per_group;                // ceil(2^64 / group); 0 for a group of 1
    int window;                                  // 0: none
    int switch_units;                            // units that stand for a segment's start and end
};

// ---------------------------------------------------------------- the split of the work
struct Request {
    int q0, nq, len;
    int nrt;           // row tiles
    int pairs;         // of row tiles, per KV head
    int P;             // units of a pair: at least the token tiles of its two row tiles, and switch_units
};

// x / group for 0 <= x < 2^32: with m = ceil(2^64 / group), x m / 2^64 exceeds x / group
// by less than x / 2^64, which is less than the 1 / group up to the next integer.
__device__ __forceinline__ int by_group(const Args& a, int x) {
    return a.group == 1 ? x : (int)__umul64hi((unsigned long long)(uint32_t)x, a.per_group);
}

// Token tiles that any row of row tile rt sees, from *first on.
template <int RT>
__device__ __forceinline__ int tiles_of(const Args& a, const Request& r, int rt, int* first) {
    const int c = r.len - r.nq;                                    // position of the first query
    int p_lo = c, p_hi = c + r.nq - 1;
    if (r.nrt > 1) {
        p_lo = c + by_group(a, rt * RT);
        p_hi = c + min(r.nq - 1, by_group(a, (rt + 1) * RT - 1));
    }
    *first = a.window ? max(0, p_lo - a.window + 1) / kTile : 0;
    return max(0, (p_hi < 0 ? 0 : p_hi / kTile + 1) - *first);
}
// The same, but at least 1: a row tile that sees nothing has its zeros to write.
template <int RT>
__device__ __forceinline__ int units_of(const Args& a, const Request& r, int rt) {
    int first;
    return max(1, tiles_of<RT>(a, r, rt, &first));
}

template <int RT>
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
    r.nrt = (r.nq * a.group + RT - 1) / RT;
    // A causal row tile has the more tokens the later it is; row tiles k and
    // nrt - 1 - k together have the same, up to one tile for the rounding (or
    // up to twice a window's tiles), so pairs are units of equal work.
    r.pairs = (r.nrt + 1) >> 1;
    r.P = 0;
    if (r.nrt == 1) r.P = units_of<RT>(a, r, 0);
    else if (r.nrt == 2 || (r.nrt > 2 && !a.window))
        r.P = units_of<RT>(a, r, 0) + units_of<RT>(a, r, r.nrt - 1) + (r.nrt > 2);
    else if (r.nrt > 2)
        r.P = 2 * min(max(1, (r.len + kTile - 1) / kTile),
                      (int)(((long long)a.window + RT / a.group + 1) / kTile) + 2);
    if (r.P) r.P += a.switch_units;
    return r;
}
// (a call holds at most kMaxUnits: the kernel checks the sum in 64 bits)
constexpr int kMaxUnits = 1 << 30;
__device__ __forceinline__ int units(const Args& a, const Request& r) { return r.pairs * r.P * a.kv_heads; }

// A chunk's share of one item (a row tile of a KV head of a request).
struct Segment {
    int b, h;            // b < 0: no more segments
    int row0, nr;        // rows of the row tile in the request's (token, head) order
    int t0, n;           // first token tile and tiles to run (0: no row sees any)
    int slot;            // -1: the whole item; else the partial's slot
    int q0, nq, len;     // the request's first row, rows and tokens
};

// The chunks of U units for n CTAs: rounds of n chunks whose sizes differ by at
// most one. Held in shared memory, for the TMA warp.
struct Chunks {
    int n, rounds;
    int at[kRounds + 1];       // first unit of each round
    int base[kRounds], rem[kRounds];

    __device__ __forceinline__ int begin(int v) const {          // first unit of chunk v; v = n * rounds: U
        const int r = (v >= n) + (v >= 2 * n);
        if (v >= n * rounds) return at[rounds];
        const int i = v - r * n;
        return at[r] + i * base[r] + min(i, rem[r]);
    }
    __device__ __forceinline__ int of(int u) const {             // the chunk that holds unit u
        const int r = (rounds > 1 && u >= at[1]) + (rounds > 2 && u >= at[2]);
        const uint32_t x = u - at[r], big = base[r] + 1, t = rem[r] * big;
        return r * n + (int)(x < t ? x / big : rem[r] + (x - t) / (uint32_t)base[r]);
    }
};

// Walks the units [u, u1) of chunk v; u is unit `off` of request b.
template <int RT>
struct Walker {
    const Chunks* ch;
    int u, u1;
    int off;
    int b, v;
    Request r;

    __device__ __forceinline__ bool next(const Args& a, Segment* s) {
        while (u < u1) {
            bool bad = false;
            while (off >= units(a, r)) {
                off -= units(a, r);
                r = request<RT>(a, ++b, &bad);
            }
            const int pair = (uint32_t)off / (uint32_t)r.P, o = off - pair * r.P;
            const int h = r.pairs == 1 ? pair : (uint32_t)pair / (uint32_t)r.pairs;
            const int k = pair - h * r.pairs;
            // the later row tile of the pair first, then the earlier, then nothing
            const int big = r.nrt - 1 - k, nb = units_of<RT>(a, r, big);
            int rt = big, at = o, n = nb;
            if (o >= nb) {
                rt = k;
                at = o - nb;
                n = k < big ? units_of<RT>(a, r, k) : 0;
            }
            if (at >= n) {
                const int skip = min(r.P - o, u1 - u);
                u += skip;
                off += skip;
                continue;
            }
            const int take = min(n - at, u1 - u);
            s->b = b;
            s->h = h;
            s->row0 = rt * RT;
            s->nr = min(RT, r.nq * a.group - s->row0);
            s->q0 = r.q0;
            s->nq = r.nq;
            s->len = r.len;
            int first;
            const int tiles = tiles_of<RT>(a, r, rt, &first);
            s->t0 = first + at;
            s->n = min(take, max(0, tiles - at));
            s->slot = -1;
            if (take != n) {
                s->slot = 2 * v + (at == 0);
                if (at == 0)       // the item goes on in the next chunks: for the join
                    a.meta[v] = make_int4((ch->of(u + n - 1) - v + 1) | (s->nr << 12) | (h << 20), r.q0, s->row0, 0);
            }
            u += take;
            off += take;
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------- small device helpers
// Barrier of the softmax threads, and one that tells them all whether any said yes.
template <int SOFT>
__device__ __forceinline__ void soft_sync() {
    asm volatile("bar.sync 1, %0;\n" ::"n"(SOFT) : "memory");
}
template <int SOFT>
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(SOFT)
        : "memory");
    return r != 0;
}
// One arrival per warp, after all its lanes (arrivals of one barrier are taken
// one by one: 512 of them held the last one up by some 1,000 cycles).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(v));
    return r;
}
// Pairs of fp32 values in one 64-bit register (one instruction for both).
using u64 = unsigned long long;
__device__ __forceinline__ u64 pack(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(u64 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
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
// Eight values times the eight factors of two 16-byte loads.
__device__ __forceinline__ void scale8(float (&v)[8], const ulonglong2& fa, const ulonglong2& fb) {
    unpack(mul2(pack(v[0], v[1]), fa.x), v[0], v[1]);
    unpack(mul2(pack(v[2], v[3]), fa.y), v[2], v[3]);
    unpack(mul2(pack(v[4], v[5]), fb.x), v[4], v[5]);
    unpack(mul2(pack(v[6], v[7]), fb.y), v[6], v[7]);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}
// One lane of the (converged) warp; the same one every time, as commits follow
// the MMAs of the thread that issued them.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
// Shared-memory descriptor of an MN-major operand in parts of PITCH = 32 or 64 bytes
// along M or N with the swizzle of that width: a row per K index, groups of 8 rows
// follow each other along K; the next part lies `part` bytes further on.
template <int PITCH>
__device__ __forceinline__ uint64_t desc_parts(uint32_t saddr, uint32_t part) {
    uint64_t d = desc_sw128(saddr, part, 8 * PITCH);
    d &= ~((uint64_t)7 << 61);
    d |= (uint64_t)(PITCH == 64 ? 4 : 6) << 61;
    return d;
}
// Two e4m3 terms of each of four values, a byte each; the second times kLoScale.
__device__ __forceinline__ void split4(float v0, float v1, float v2, float v3, uint32_t* hi, uint32_t* lo) {
    const __half2 a = __floats2half2_rn(v0, v1), b = __floats2half2_rn(v2, v3);
    const uint32_t ha = __nv_cvt_halfraw2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hb = __nv_cvt_halfraw2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    __half2 ra = __hsub2(a, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)ha, __NV_E4M3)));
    __half2 rb = __hsub2(b, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hb, __NV_E4M3)));
    const __half2 f = __float2half2_rn(kLoScale);
    ra = __hmul2(ra, f);
    rb = __hmul2(rb, f);
    const uint32_t la = __nv_cvt_halfraw2_to_fp8x2(ra, __NV_SATFINITE, __NV_E4M3);
    const uint32_t lb = __nv_cvt_halfraw2_to_fp8x2(rb, __NV_SATFINITE, __NV_E4M3);
    *hi = ha | (hb << 16);
    *lo = la | (lb << 16);
}
// Three e5m2 terms of each of four values >= 0 (rounded to fp16 first), a byte each. An
// e5m2 code is the upper byte of an fp16 value: the first two terms are cut off, which
// leaves exact remainders, the third is rounded to nearest. Together they are within 2^-9
// (or 2^-17) of the value. (All three rounded hold fp16 exactly, for four more conversions:
// the prompt chunk 634 us; this way 592.)
__device__ __forceinline__ void split4_e5m2(float v0, float v1, float v2, float v3, uint32_t (&out)[3]) {
    __half2 a = __floats2half2_rn(v0, v1), b = __floats2half2_rn(v2, v3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t wa, wb;
        memcpy(&wa, &a, 4);
        memcpy(&wb, &b, 4);
        out[i] = __byte_perm(wa, wb, 0x7531);
        wa &= 0xff00ff00u;
        wb &= 0xff00ff00u;
        __half2 ca, cb;
        memcpy(&ca, &wa, 4);
        memcpy(&cb, &wb, 4);
        a = __hsub2(a, ca);
        b = __hsub2(b, cb);
    }
    out[2] = __nv_cvt_halfraw2_to_fp8x2(a, __NV_SATFINITE, __NV_E5M2) |
             (uint32_t)__nv_cvt_halfraw2_to_fp8x2(b, __NV_SATFINITE, __NV_E5M2) << 16;
}

constexpr int kSegs = 4;     // segments handed on ahead of their use
constexpr int kScales = 8;   // token tiles whose block scales are held: more than the ring holds tiles

template <typename S>
struct Bars {
    uint64_t full[S::SLOTS];     // a block's bytes landed
    uint64_t empty[S::SLOTS];    // the MMAs that read it completed
    uint64_t seg_full[kSegs];    // a segment is written
    uint64_t seg_empty[kSegs];   // the MMA warp and the softmax warps have done with it
    uint64_t sc_full[kScales];   // a tile's block scales are written
    uint64_t q_full;             // the queries are in shared memory
    uint64_t s_full;             // S^T of a tile is in TMEM
    uint64_t s_free;             // the softmax warps have it in registers
    uint64_t p_full;             // the weights are in shared memory (and O^T is rescaled)
    uint64_t pv_done;            // PV completed
    uint64_t drain;
    long long warp_sums[33];
    int before[S::THREADS];           // units before each thread's requests
    Chunks ch;
    uint32_t tmem_base;
    int abort;
    alignas(16) float4 sc[kScales][8];   // (ks, log2 vs, 1 / vs) of a tile's blocks
    // of each row; what the outputs of a segment still need while the next begins, twice
    alignas(16) float nref[2][S::RT]; // minus the reference exponent
    alignas(16) float fac[S::RT];     // 2^(old reference - new)
    alignas(16) float qs[S::RT];      // query scale * softmax scale * log2 e
    float part[4][S::RT];             // per-warp maxima, then sums
    float sum[S::RT];
    // of each segment handed on: rows' (row of q and out, head) and tokens' positions (-1: no row)
    alignas(16) int2 row[kSegs][S::RT];
    alignas(16) int pos[kSegs][S::RT];
    int2 span[kSegs];                 // positions of the first and the last row
    Segment seg[kSegs];
};

template <typename S>
constexpr int smem_bytes() {
    return S::kOffBars + (int)sizeof(Bars<S>) + 1024;
}

// The sums over a warp of 16 columns: lane i writes column i.
__device__ __forceinline__ void column_sums(float (&v)[16], int lane, float* out) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = lane & o;
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    if (lane < 16) out[lane] = v[0];
}

// ---------------------------------------------------------------- the kernel
template <typename S>
__global__ void __launch_bounds__(S::THREADS, S::CTAS)
attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
              const __grid_constant__ Args a) {
    constexpr int DB = S::DB, RT = S::RT, N = S::N, CT = S::CT, SOFT = S::SOFT;
    constexpr int kWarpTma = SOFT / 32, kWarpMma = kWarpTma + 1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Bars<S>& bs = *reinterpret_cast<Bars<S>*>(sm + S::kOffBars);
    volatile int* abort = &bs.abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_grid = gridDim.x, cta = blockIdx.x;

    // ------------------------------------------------------------ the units
    // Prefix sums over the requests: of a few by the TMA warp alone while the others
    // set up, of many by every thread.
    const int per = (a.n_req + S::THREADS - 1) / S::THREADS;       // requests per thread (at most 22)
    const bool few = a.n_req <= 32;
    bool bad = false;
    if (warp == kWarpTma && lane == 0) {
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(&kmap) : "memory");
        if (!S::SHARED) asm volatile("prefetch.tensormap [%0];\n" ::"l"(&vmap) : "memory");
    }
    if (!few || warp == kWarpTma) {
        const int i = few ? lane : tid;
        const int b0 = min(a.n_req, i * per), b1 = min(a.n_req, b0 + per);
        long long mine = 0, incl, total;
        for (int b = b0; b < b1; ++b) {
            const Request r = request<RT>(a, b, &bad);
            mine += (long long)r.pairs * r.P * a.kv_heads;
            // where cu descends, requests may share rows of out: refused like too much work
            if (a.cu[b + 1] < a.cu[b]) mine += 2ll * kMaxUnits;
        }
        if (few) {
            incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            total = __shfl_sync(0xffffffffu, incl, 31);
        } else {
            incl = block_scan(mine, bs.warp_sums, &total);
        }
        if (cta == 0 && bad) atomicOr(a.err, kErrBounds);
        if (total > kMaxUnits) {                           // reported, nothing written
            if (i == 0) atomicOr(a.err, kErrBounds);
            total = 0;
        }
        // as few CTAs as keep the largest share the same: fewer parts to join
        const int U = (int)total, most = (U + n_grid - 1) / n_grid;
        const int n_cta = U ? (U + most - 1) / most : 0;
        // rounds of smaller chunks only where their switches are few beside their units: from
        // about 200 per CTA on (the prompt chunk, with 400: 593 us, 629 without; decode of
        // 256-dim heads with 220: 683 and 687; of 128-dim heads with 245 710 and 713, with 113
        // 389 and 386, with 85 301 and 292)
        const int rounds = S::ROUNDS > 1 && U / kRoundsFrom >= n_cta ? S::ROUNDS : 1;
        bs.before[i] = (int)(incl - mine);
        if (i == 0) {
            bs.ch.n = n_cta;
            bs.ch.rounds = rounds;
            if (cta == 0) a.ctrl[1] = n_cta * rounds;
        }
        if (i <= kRounds && cta < n_cta) {
            auto begin = [&](int r) { return rounds == 1 ? (r ? U : 0) : (int)((long long)U * cut(r) / 16); };
            const int at = begin(i);
            bs.ch.at[i] = at;
            if (i < kRounds) {
                const uint32_t n = begin(i + 1) - at;
                bs.ch.base[i] = n / (uint32_t)n_cta;
                bs.ch.rem[i] = n % (uint32_t)n_cta;
            }
        }
    }
    if (tid == 0) {
        for (int s = 0; s < S::SLOTS; ++s) {
            mbar_init(&bs.full[s], 1);
            mbar_init(&bs.empty[s], 1);
        }
        for (int k = 0; k < kSegs; ++k) {
            mbar_init(&bs.seg_full[k], 1);
            mbar_init(&bs.seg_empty[k], 2);
        }
        for (int k = 0; k < kScales; ++k) mbar_init(&bs.sc_full[k], 1);
        mbar_init(&bs.q_full, SOFT / 32);
        mbar_init(&bs.s_full, 1);
        mbar_init(&bs.s_free, SOFT / 32);
        mbar_init(&bs.p_full, SOFT / 32);
        mbar_init(&bs.pv_done, 1);
        mbar_init(&bs.drain, 1);
        bs.abort = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) tmem_alloc(&bs.tmem_base, S::ALLOC);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bs.tmem_base;
    if (cta >= bs.ch.n) {                                  // nothing to do (every thread)
        if (warp == kWarpMma) tmem_dealloc(tmem, S::ALLOC);
        return;
    }
    const uint32_t tm_s = tmem, tm_o = tmem + N;

    bool ok = true;
    if (warp == kWarpTma) {
        // ======================================================== TMA
        // Also walks the CTA's units and hands its segments on, and brings the block
        // scales of each token tile (the tile's few blocks, a lane each).
        Segment sg{};
        Walker<RT> w;
        const Chunks& ch = bs.ch;
        w.ch = &ch;
        // to the first unit of chunk v
        auto seek = [&](int v) {
            w.v = v;
            w.u = ch.begin(v);
            w.u1 = ch.begin(v + 1);
            int lo = 0, hi = min(a.n_req, S::THREADS);
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (bs.before[mid] <= w.u) lo = mid;
                else hi = mid;
            }
            // the last thread at or below u owns it (threads without units have the next one's sum)
            const int b0 = lo * per, rel = w.u - bs.before[lo];
            w.b = b0;
            w.off = rel;
            if (per > 1) {
                const int b = b0 + lane;
                const int k = lane < per && b < a.n_req ? units(a, request<RT>(a, b, &bad)) : 0;
                int incl = k;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                const int mine = __ffs(__ballot_sync(0xffffffffu, rel < incl)) - 1;
                w.b = b0 + mine;
                w.off = rel - __shfl_sync(0xffffffffu, incl - k, mine);
            }
            w.r = request<RT>(a, w.b, &bad);
            if (lane == 0) a.meta[v] = make_int4(0, 0, 0, 0);      // no item goes on from this chunk, so far
            __syncwarp();
        };
        seek(cta);
        uint32_t it = 0, g = 0;                            // blocks of 128 dims requested, token tiles
        bool ids_bad = false;
        const int bpt = kTile >> a.bs_log2, bsz = 1 << a.bs_log2;
        auto id_at = [&](int tile) -> int {                // this lane's block of a tile (-1: none there)
            const int at = tile * bpt + lane;
            if (lane >= bpt || at * bsz >= sg.len) return -1;
            const int id = __ldg(a.table + (size_t)sg.b * a.max_blocks + at);
            // an id that is no block reads as zeros (out of the tensor's range)
            if (id >= 0 && id < a.n_blocks) return id;
            ids_bad = true;
            return a.n_blocks;
        };
        auto load = [&](int id, bool is_v) -> bool {
            const int nb = __popc(__ballot_sync(0xffffffffu, id >= 0));
            for (int d = 0; d < DB; ++d) {
                const int s = it % S::SLOTS;
                const bool got = it < S::SLOTS || mbar_wait_abort(&bs.empty[s], ((it / S::SLOTS) + 1) & 1, abort) > 0;
                if (!__all_sync(0xffffffffu, got)) return false;
                if (lane == 0) mbar_arrive_expect_tx(&bs.full[s], (uint32_t)(nb * bsz * 128));
                __syncwarp();
                if (lane < nb)
                    tma_load_4d(smem_u32(sm + s * kSlotBytes) + lane * bsz * 128, is_v ? &vmap : &kmap, d * 128, 0, sg.h, id,
                                &bs.full[s]);
                ++it;
            }
            return true;
        };
        for (uint32_t k = 0; ok; ++k) {
            bool more = w.next(a, &sg);
            while (!more && ch.rounds > 1) {               // the next chunk that nobody has
                int v = 0;
                if (lane == 0) v = ch.n + atomicAdd(a.ctrl, 1);
                v = __shfl_sync(0xffffffffu, v, 0);
                if (v >= ch.n * ch.rounds) break;
                seek(v);
                more = w.next(a, &sg);
            }
            const bool got = k < kSegs || mbar_wait_abort(&bs.seg_empty[k % kSegs], ((k / kSegs) + 1) & 1, abort) > 0;
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            if (!more) {
                sg.b = -1;
                sg.n = 0;
            }
            if (more) {
                // its rows, here, where no one waits for the divisions
                for (int r = lane; r < RT; r += 32) {
                    const bool on = r < sg.nr;
                    const int row = sg.row0 + r, qt = on ? by_group(a, row) : 0, p = sg.len - sg.nq + qt;
                    bs.row[k % kSegs][r] = make_int2(sg.q0 + qt, sg.h * a.group + (on ? row - qt * a.group : 0));
                    bs.pos[k % kSegs][r] = on ? p : -1;
                    if (r == 0) bs.span[k % kSegs].x = p;
                    if (r == sg.nr - 1) bs.span[k % kSegs].y = p;
                }
                __syncwarp();
            }
            if (lane == 0) {
                bs.seg[k % kSegs] = sg;
                mbar_arrive(&bs.seg_full[k % kSegs]);
            }
            __syncwarp();
            if (!more) break;
            int id = sg.n > 0 ? id_at(sg.t0) : -1, id_v = -1;
            for (int j = 0; ok && j < sg.n; ++j, ++g) {
                const int id_next = j + 1 < sg.n ? id_at(sg.t0 + j + 1) : -1;
                float ks = 0.f, vs = 0.f;
                const bool there = id >= 0 && id < a.n_blocks;
                if (there) {
                    const size_t at = (size_t)id * a.kv_heads + sg.h;
                    ks = __ldg(a.ks + at);
                    vs = S::SHARED ? ks : __ldg(a.vs + at);
                }
                ok = load(id, false);
                if (!ok) break;
                // (tile g - kScales was read before the slot just taken came free)
                vs = vs < 5.421010862427522e-20f ? 5.421010862427522e-20f : vs;   // 2^-64: a scale of 0 too
                if (lane < bpt)
                    bs.sc[g % kScales][lane] = there ? make_float4(ks, lg2(vs), __fdividef(1.f, vs), 0.f)
                                                     : make_float4(0.f, -INFINITY, 0.f, 0.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bs.sc_full[g % kScales]);
                if (!S::SHARED && j > 0) ok = load(id_v, true);
                id_v = id;
                id = id_next;
            }
            if (!S::SHARED && ok && sg.n > 0) ok = load(id_v, true);
        }
        if (ids_bad) atomicOr(a.err, kErrBounds);
        if (!ok)   // every copy issued lands before the CTA may leave
            for (uint32_t i = it > S::SLOTS ? it - S::SLOTS : 0; i < it; ++i)
                mbar_wait(&bs.full[i % S::SLOTS], (i / S::SLOTS) & 1);
    } else if (warp == kWarpMma) {
        // ======================================================== MMA issue
        // The whole warp walks and waits, one elected lane issues: descriptors then
        // stay in uniform registers (a lane of its own took 58 cycles per MMA to
        // issue, this way 40; N = 64 and 128 run at 48 and 64, the rate at which
        // their operands leave shared memory).
        constexpr uint32_t id_qk = idesc_f32acc(0, 0, 0, kTile, N);              // e4m3, both K-major
        constexpr uint32_t id_pv = idesc_f32acc(0, 1, 1, 128, S::ON) | (1u << 10);   // both MN-major, B is e5m2
        constexpr uint32_t id_two = idesc_f32acc(0, 1, 1, 128, 2 * RT) | (1u << 10);
        const uint32_t r0 = smem_u32(sm);
        const uint64_t qd = desc_sw128(smem_u32(sm + S::kOffQ), 16, 1024);
        const uint64_t pd = desc_parts<S::kPitch>(smem_u32(sm + S::kOffP), S::kPart);
        uint32_t it = 0, g = 0, segs = 0;                  // blocks taken, token tiles, segments with tiles
        auto got = [&](uint64_t* bar, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait_abort(bar, parity, abort) > 0);
        };
        // PV of tile gt, whose K blocks began at block `k_it` of the ring
        auto pv = [&](uint32_t gt, bool first, uint32_t k_it) -> bool {
            if (!got(&bs.p_full, gt & 1)) return false;
#pragma unroll
            for (int mb = 0; mb < DB; ++mb) {
                const uint32_t i = S::SHARED ? k_it + mb : it + mb, s = i % S::SLOTS;
                if (!S::SHARED && !got(&bs.full[s], (i / S::SLOTS) & 1)) return false;
                tc_fence_after();
                const uint64_t vd = desc_sw128(r0 + s * kSlotBytes, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 32; ++kk) {
                        const uint64_t ad = vd + kk * (32 * 128 / 16);
                        const uint32_t o = tm_o + S::o_at(mb);
                        mma_f8(o, ad, pd + kk * (32 * S::kPitch / 16), mb < S::TWO ? id_two : id_pv, !first || kk > 0);
                        if (!S::CAT) {
#pragma unroll
                            for (int i = mb < S::TWO ? 2 : 1; i < 3; ++i)
                                mma_f8(o, ad, pd + (i * S::kPart + kk * 32 * S::kPitch) / 16, id_pv, 1);
                        }
                    }
                    mma_commit(&bs.empty[s]);
                    if (mb == DB - 1) mma_commit(&bs.pv_done);
                }
                __syncwarp();
            }
            if (!S::SHARED) it += DB;
            return true;
        };
        for (uint32_t k = 0; ok; ++k) {
            ok = got(&bs.seg_full[k % kSegs], (k / kSegs) & 1);
            if (!ok) break;
            const int n = bs.seg[k % kSegs].n;
            const bool last = bs.seg[k % kSegs].b < 0;
            warp_arrive(&bs.seg_empty[k % kSegs], lane);
            if (last) break;
            if (n == 0) continue;
            ok = got(&bs.q_full, segs & 1);
            ++segs;
            uint32_t k_it = 0;
            for (int j = 0; ok && j < n; ++j) {
                if (g > 0) ok = got(&bs.s_free, (g - 1) & 1);
                const uint32_t k_new = it;
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const uint32_t s = (it + d) % S::SLOTS;
                    if (!ok || !got(&bs.full[s], ((it + d) / S::SLOTS) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t kd = desc_sw128(r0 + s * kSlotBytes, 16, 1024);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8(tm_s, kd + kk * 2, qd + (d * N * 128 + kk * 32) / 16, id_qk, (d | kk) != 0);
                        if (!S::SHARED) mma_commit(&bs.empty[s]);
                        if (d == DB - 1) mma_commit(&bs.s_full);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                it += DB;
                ++g;
                if (j > 0) ok = pv(g - 2, j == 1, k_it);
                k_it = k_new;
            }
            if (ok) ok = pv(g - 1, n == 1, k_it);
        }
        // every MMA issued completes before TMEM is freed
        if (elect_one()) mma_commit(&bs.drain);
        __syncwarp();
        if (!mbar_wait(&bs.drain, 0)) ok = false;
    } else {
        // ======================================================== softmax
        const int quad = warp & 3, col0 = (warp >> 2) * CT;    // TMEM lanes of this warp, first column
        const int tok = quad * 32 + lane;                      // token of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t my_s = tm_s + lane_base + col0, my_o = tm_o + lane_base + col0;
        unsigned char* qsm = sm + S::kOffQ;
        unsigned char* psm = sm + S::kOffP;
        uint32_t g = 0, it = 0;                            // token tiles, blocks of the ring
        bool fail = false;
        u64 l2[CT / 2];                                    // sums of p / vs, two rows each
        // queries: a warp per row, 4 values per lane and 128 dims
        constexpr int W = SOFT / 32, RPW = RT / W;
        uint2 qx[RPW][DB];
        auto load_q = [&](const Segment& sg, uint32_t k) {
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int r = warp + W * i;
                const int2 at = bs.row[k % kSegs][r];
                const uint16_t* p = a.q + (size_t)at.x * a.q_row + (size_t)at.y * (DB * 128) + lane * 4;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    qx[i][d] = r < sg.nr ? __ldg(reinterpret_cast<const uint2*>(p + d * 128)) : make_uint2(0, 0);
            }
        };
        // Segment k's rows into shared memory, the queries from the registers.
        auto stage = [&](const Segment& sg, uint32_t k) {
            if (tid < RT) {
                // a column without a row is held at weight 0 by a reference out of reach
                bs.nref[k & 1][tid] = tid < sg.nr ? -kLow : kLow;
            }
            if (sg.n == 0) return;
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int r = warp + W * i;
                uint32_t m = 0;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    m = max(m, max(max(qx[i][d].x & 0x7fffu, (qx[i][d].x >> 16) & 0x7fffu),
                                   max(qx[i][d].y & 0x7fffu, (qx[i][d].y >> 16) & 0x7fffu)));
                m = __reduce_max_sync(0xffffffffu, m);
                const int e = min(max((int)(m >> 7) - 127 - 7, -120), 120);
                const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
                if (lane == 0)   // a row that is not finite has no result: NaN
                    bs.qs[r] = m >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                            : __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    uint32_t hi, lo;
                    split4(__uint_as_float(qx[i][d].x << 16) * inv, __uint_as_float(qx[i][d].x & 0xffff0000u) * inv,
                           __uint_as_float(qx[i][d].y << 16) * inv, __uint_as_float(qx[i][d].y & 0xffff0000u) * inv,
                           &hi, &lo);
                    unsigned char* q = qsm + d * (N * 128) + (lane & 3) * 4;
                    *reinterpret_cast<uint32_t*>(q + sw128(r, lane >> 2)) = hi;
                    *reinterpret_cast<uint32_t*>(q + sw128(RT + r, lane >> 2)) = lo;
                }
            }
            fence_async_smem();
            warp_arrive(&bs.q_full, lane);
        };
        // (what a warp does after a failed wait, all its lanes do: collectives follow)
        auto warp_got = [&](uint64_t* bar, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait_abort(bar, parity, abort) > 0);
        };
        if (RT == 16)   // the fourth columns of 16-row tiles, for good (before the first weights' fence)
            *reinterpret_cast<uint4*>(psm + S::p_at(tok, 3)) = make_uint4(0, 0, 0, 0);
        if (!warp_got(&bs.seg_full[0], 0)) fail = true;
        else {
            if (bs.seg[0].n > 0) load_q(bs.seg[0], 0);
            if (bs.seg[0].b >= 0) stage(bs.seg[0], 0);
        }
        for (uint32_t k = 0;; ++k) {
            const Segment& sg = bs.seg[k % kSegs];
            if (soft_any<SOFT>(fail)) {                    // also: the rows are staged
                ok = false;
                break;
            }
            if (k > 0 && tid == 0) mbar_arrive(&bs.seg_empty[(k - 1) % kSegs]);
            if (sg.b < 0) break;
            const int n = sg.n, len = sg.len;
            float* const nref = bs.nref[k & 1];
#pragma unroll
            for (int c = 0; c < CT / 2; ++c) l2[c] = 0;
            bool stop = false;
            for (int j = 0; j < n; ++j, ++g) {
                const int t0 = (sg.t0 + j) * kTile, t = t0 + tok;
                if (mbar_wait_abort(&bs.s_full, g & 1, abort) <= 0 ||
                    mbar_wait_abort(&bs.sc_full[g % kScales], (g / kScales) & 1, abort) <= 0)
                    fail = true;
                const float4 sc = bs.sc[g % kScales][tok >> a.bs_log2];   // (0, -inf, 0) without a block
                tc_fence_after();
                const int win = a.window ? a.window : 1 << 30;
                const int2 span = bs.span[k % kSegs];
                const bool edge = t0 + kTile - 1 > span.x || t0 <= span.y - win;
                const u64 ks2 = pack(sc.x, sc.x), lv2 = pack(sc.y, sc.y);
                // exponents: score * log2 e + log2 vs, -inf where not seen
                float x[CT], most = kLow;
                {
                    float lo[CT];
                    tmem_ld16(my_s, x);
                    tmem_ld16(my_s + RT, lo);
                    tmem_ld_wait();
                    tmem_regs_ready(x);
                    tmem_regs_ready(lo);
                    tc_fence_before();
                    warp_arrive(&bs.s_free, lane);
                    const u64 lo_f = pack(1.f / kLoScale, 1.f / kLoScale);
#pragma unroll
                    for (int i = 0; i < CT; i += 4) {
                        const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(&bs.qs[col0 + i]);
                        const u64 a0 = fma2(pack(lo[i], lo[i + 1]), lo_f, pack(x[i], x[i + 1]));
                        const u64 a1 = fma2(pack(lo[i + 2], lo[i + 3]), lo_f, pack(x[i + 2], x[i + 3]));
                        unpack(fma2(mul2(a0, s4.x), ks2, lv2), x[i], x[i + 1]);
                        unpack(fma2(mul2(a1, s4.y), ks2, lv2), x[i + 2], x[i + 3]);
                    }
                }
                if (edge) {
#pragma unroll
                    for (int i = 0; i < CT; ++i) {
                        const int p = bs.pos[k % kSegs][col0 + i];
                        if (t > p || t <= p - win) x[i] = -INFINITY;
                    }
                }
                // the same relative to the rows' references, now
                auto above = [&](float (&y)[CT]) {
#pragma unroll
                    for (int i = 0; i < CT; i += 4) {
                        const ulonglong2 r4 = *reinterpret_cast<const ulonglong2*>(&nref[col0 + i]);
                        unpack(add2(pack(x[i], x[i + 1]), r4.x), y[i], y[i + 1]);
                        unpack(add2(pack(x[i + 2], x[i + 3]), r4.y), y[i + 2], y[i + 3]);
                    }
                };
                float y[CT];
                if (j > 0) {
                    above(y);
#pragma unroll
                    for (int i = 0; i < CT; i += 2) most = max3(most, y[i], y[i + 1]);
                }
                if (j == 0 || soft_any<SOFT>(most > kRoom || fail)) {
                    // new references: the maximum of the tile's 128 tokens per row
                    float m = -INFINITY;
#pragma unroll
                    for (int i = 0; i < CT; ++i) {
                        const float mc = warp_max(x[i]);
                        if (lane == i) m = mc;
                    }
                    if (lane < CT) bs.part[quad][col0 + lane] = m;
                    if (soft_any<SOFT>(fail)) {            // the same answer for every softmax thread
                        stop = true;
                        break;
                    }
                    if (tid < RT) {
                        const float mt = fmaxf(fmaxf(bs.part[0][tid], bs.part[1][tid]), fmaxf(bs.part[2][tid], bs.part[3][tid]));
                        const float was = -nref[tid];
                        float now = was;
                        if (mt - was > kHead) now = mt - kHead;     // every row that grew, while at it
                        nref[tid] = -now;
                        bs.fac[tid] = now == was ? 1.f : ex2(was - now);
                    }
                    soft_sync<SOFT>();
                    if (j > 0) {
                        if (mbar_wait_abort(&bs.pv_done, (g - 1) & 1, abort) <= 0) fail = true;
                        tc_fence_after();
                    }
                    // sums and outputs of the 8 rows around one that moved
#pragma unroll
                    for (int c = 0; c < CT; c += 8) {
                        const ulonglong2 fa = *reinterpret_cast<const ulonglong2*>(&bs.fac[col0 + c]);
                        const ulonglong2 fb = *reinterpret_cast<const ulonglong2*>(&bs.fac[col0 + c + 4]);
                        const u64 one = pack(1.f, 1.f);
                        if (fa.x == one && fa.y == one && fb.x == one && fb.y == one) continue;
                        l2[c / 2] = mul2(l2[c / 2], fa.x);
                        l2[c / 2 + 1] = mul2(l2[c / 2 + 1], fa.y);
                        l2[c / 2 + 2] = mul2(l2[c / 2 + 2], fb.x);
                        l2[c / 2 + 3] = mul2(l2[c / 2 + 3], fb.y);
                        if (j == 0) continue;
                        // pieces of 8 columns, RT apart: the three terms of 128 dims, or any two
                        constexpr int KP = S::CAT ? 3 : 2, GROUPS = S::CAT ? DB : (DB + S::TWO) / 2;
#pragma unroll 1
                        for (int i0 = 0; i0 < GROUPS; ++i0) {
                            const uint32_t at = my_o + i0 * (S::CAT ? S::ON : 2 * RT) + c;
                            float o[KP][8];
#pragma unroll
                            for (int i = 0; i < KP; ++i) tmem_ld<8>(at + i * RT, o[i]);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < KP; ++i) {
                                tmem_regs_ready_n<8>(o[i]);
                                scale8(o[i], fa, fb);
                                tmem_st<8>(at + i * RT, o[i]);
                            }
                        }
                    }
                    if (j > 0) {
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    above(y);
                }
                const u64 iv2 = pack(sc.z, sc.z);
                // the weights of the last tile have been read
                if (g > 0 && mbar_wait_abort(&bs.pv_done, (g - 1) & 1, abort) <= 0) fail = true;
                {
                    uint32_t w[3][4];
#pragma unroll
                    for (int i = 0; i < CT; i += 4) {
                        const float v0 = ex2(y[i]), v1 = ex2(y[i + 1]), v2 = ex2(y[i + 2]), v3 = ex2(y[i + 3]);
                        l2[i / 2] = fma2(pack(v0, v1), iv2, l2[i / 2]);
                        l2[i / 2 + 1] = fma2(pack(v2, v3), iv2, l2[i / 2 + 1]);
                        uint32_t term[3];
                        split4_e5m2(v0, v1, v2, v3, term);
#pragma unroll
                        for (int k = 0; k < 3; ++k) w[k][i / 4] = term[k];
                    }
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        *reinterpret_cast<uint4*>(psm + S::p_at(tok, i * S::CG + col0 / 16)) =
                            make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                }
                if (t0 + kTile > len) {
                    // rows behind the request: whatever lies there must not meet a weight of 0 as NaN
                    // (the request's last tile, so the last of the segment: its V blocks end the segment's)
                    const uint32_t v0 = it + (S::SHARED ? n - 1 : 2 * n - 1) * DB;
                    for (int d = 0; d < DB; ++d) {
                        const uint32_t s = (v0 + d) % S::SLOTS;
                        if (mbar_wait_abort(&bs.full[s], ((v0 + d) / S::SLOTS) & 1, abort) <= 0) fail = true;
                        if (t >= len)
                            for (int i = warp >> 2; i < 8; i += S::CG)
                                *reinterpret_cast<uint4*>(sm + s * kSlotBytes + tok * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                warp_arrive(&bs.p_full, lane);
            }
            if (stop) {
                ok = false;
                break;
            }
            it += n * (S::SHARED ? DB : 2 * DB);
            // the next segment's queries, so that its first product runs during the outputs
            const Segment& next = bs.seg[(k + 1) % kSegs];
            bool go = false;
            if (!warp_got(&bs.seg_full[(k + 1) % kSegs], ((k + 1) / kSegs) & 1)) fail = true;
            else go = next.b >= 0;
            if (go && next.n > 0) load_q(next, k + 1);
            if (n > 0) {
                float l[CT];
#pragma unroll
                for (int c = 0; c < CT; c += 2) unpack(l2[c / 2], l[c], l[c + 1]);
                column_sums(l, lane, &bs.part[quad][col0]);
            }
            soft_sync<SOFT>();                             // every warp is through with this segment's rows
            if (go) stage(next, k + 1);
            const int slot = sg.slot, nr = sg.nr;
            if (tid < RT) {
                const float sum = n > 0 ? (bs.part[0][tid] + bs.part[1][tid]) + (bs.part[2][tid] + bs.part[3][tid]) : 0.f;
                bs.sum[tid] = sum == 0.f ? 0.f : 1.f / sum;
                if (slot >= 0)
                    reinterpret_cast<float2*>(a.part_ml)[(size_t)slot * RT + tid] = make_float2(-nref[tid], sum);
            }
            // ---------------------------------------------------- out
            if (n > 0) {
                if (mbar_wait_abort(&bs.pv_done, (g - 1) & 1, abort) <= 0) fail = true;
                tc_fence_after();
            }
            soft_sync<SOFT>();
            // (a part without tiles has the sum 0, by which the join leaves it out)
            if (n > 0 || slot < 0) {
#pragma unroll
                for (int c = 0; c < CT; c += 8) {
                    const int rows = min(8, nr - col0 - c);
                    if (rows <= 0) break;
                    float inv[8];
                    uint16_t* at[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        inv[i] = bs.sum[col0 + c + i];
                        const int2 row = bs.row[k % kSegs][col0 + c + i];
                        at[i] = a.out + (size_t)row.x * a.out_row + (size_t)row.y * (DB * 128) + tok;
                    }
                    float* po = a.part_o + ((size_t)max(slot, 0) * RT + col0 + c) * (DB * 128) + tok;
#pragma unroll 1
                    for (int mb = 0; mb < DB; ++mb) {
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = 0.f;
                        if (n > 0) {
                            tmem_ld<8>(my_o + S::o_at(mb) + c, o);
                            if (S::CAT || mb < S::TWO) {
                                float o2[8];
                                tmem_ld<8>(my_o + S::o_at(mb) + RT + c, o2);
                                tmem_ld_wait();
                                tmem_regs_ready_n<8>(o);
                                tmem_regs_ready_n<8>(o2);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] += o2[i];
                                if (S::CAT) {
                                    tmem_ld<8>(my_o + S::o_at(mb) + 2 * RT + c, o2);
                                    tmem_ld_wait();
                                    tmem_regs_ready_n<8>(o2);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) o[i] += o2[i];
                                }
                            } else {
                                tmem_ld_wait();
                                tmem_regs_ready_n<8>(o);
                            }
                        }
                        if (slot < 0) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (i < rows)
                                    at[i][mb * 128] = __bfloat16_as_ushort(__float2bfloat16_rn(inv[i] == 0.f ? 0.f : o[i] * inv[i]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (i < rows) po[i * (DB * 128) + mb * 128] = o[i];
                        }
                    }
                }
                tc_fence_before();
            }
        }
        if (fail) ok = false;
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    const bool failed = __syncthreads_or(!ok);
    if (failed && tid == 0) atomicOr(a.err, kErrTimeout);
    pdl_trigger();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, S::ALLOC);
    }
}

// ---------------------------------------------------------------- joining split items
// Row r of a split item: its parts' references m_i and sums l_i give weights
// 2^(m_i - max m); out = sum w_i O_i / sum w_i l_i, in part order. A job is 128
// dims of one row: 4 per lane of a warp. Items of few parts give a warp a job
// each; of an item of many (one long request), a CTA's warps share a job's
// parts and add up in warp order. Latency-bound: a chain of three loads.
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFewParts = 12;
constexpr int kMaxChunks = 1920;   // 4 CTAs x 160 SMs x 3 rounds; a part count fits 12 bits

// Weighted sum of parts [p0, p1) for 4 dims per lane; every lane gets sum w_i l_i.
template <int RT>
__device__ __forceinline__ float4 join_parts(const Args& a, int v0, int parts, int row, int dims, int d, int p0, int p1,
                                             float m, float* sum_out) {
    const int lane = threadIdx.x & 31;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    // part i's slot: the first chunk's trailing segment, the others' leading one
    auto slot = [&](int i) { return (size_t)(2 * (v0 + i) + (i == 0)); };
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int base = p0; base < p1; base += 32) {
        float w = 0.f;
        if (base + lane < p1) {
            const float2 v = __ldcg(&ml[slot(base + lane) * RT + row]);
            if (v.y != 0.f) {                              // a part with no weight is not read
                w = ex2(v.x - m);
                sum = fmaf(w, v.y, sum);
            }
        }
        const int n = min(32, p1 - base);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float f = __shfl_sync(0xffffffffu, w, i);
            if (f == 0.f) continue;
            const float4 o = __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot(base + i) * RT + row) * dims + d) + lane);
            acc.x = fmaf(f, o.x, acc.x);
            acc.y = fmaf(f, o.y, acc.y);
            acc.z = fmaf(f, o.z, acc.z);
            acc.w = fmaf(f, o.w, acc.w);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    *sum_out = sum;
    return acc;
}

template <int DB, int RT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args a) {
    __shared__ long long warp_sums[33];
    // split items: (parts | rows << 12 | KV head << 20, first row of out, row, chunk it begins in)
    __shared__ int4 item[kMaxChunks];
    __shared__ int first[kMaxChunks + 1];             // CTA jobs before each
    __shared__ float4 acc_s[kJoinWarps][32];
    __shared__ float sum_s[kJoinWarps], max_s[kJoinWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    const int n_chunks = min(a.ctrl[1], kMaxChunks);
    if (blockIdx.x == 0 && tid == 0) a.ctrl[0] = 0;   // for the next call
    int n_items = 0, n_jobs = 0;
    for (int base = 0; base < n_chunks; base += kJoinThreads) {
        const int i = base + tid;
        int4 it = i < n_chunks ? __ldcg(&a.meta[i]) : make_int4(0, 0, 0, 0);
        int parts = it.x & 0xfff;
        const int nr = (it.x >> 12) & 0xff, jobs = nr * DB;
        // (when every CTA gave up on a wait, chunks nobody took still hold an earlier call's items)
        if (nr > RT || (it.x >> 20) >= a.kv_heads || parts > n_chunks - i || it.y + (it.z + nr - 1) / a.group >= a.n_rows)
            parts = 0;
        const int cta_jobs = parts <= kFewParts ? (jobs + kJoinWarps - 1) / kJoinWarps : jobs;
        // items in the high half, jobs in the low one
        long long total;
        const long long incl = block_scan(parts ? (1ll << 32) + cta_jobs : 0, warp_sums, &total);
        if (parts) {
            const int k = n_items + (int)(incl >> 32) - 1;
            it.w = i;
            item[k] = it;
            first[k] = n_jobs + (int)(incl & 0xffffffff) - cta_jobs;
        }
        n_items += (int)(total >> 32);
        n_jobs += (int)(total & 0xffffffff);
    }
    __syncthreads();
    for (int job = blockIdx.x; job < n_jobs; job += gridDim.x) {
        const int k = last_not_above(first, n_items, job);
        const int4 it = item[k];
        const int parts = it.x & 0xfff, nr = (it.x >> 12) & 0xff, v0 = it.w;
        const bool shared_job = parts > kFewParts;
        const int j = shared_job ? job - first[k] : (job - first[k]) * kJoinWarps + warp;
        if (j >= nr * DB) continue;                   // a warp without a job (never in a shared one)
        const int row = j / DB, d = (j - row * DB) * 128;
        float m = kLow;
        auto see = [&](int i) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + (size_t)(2 * (v0 + i) + (i == 0)) * RT + row);
            if (v.y != 0.f) m = fmaxf(m, v.x);
        };
        if (shared_job) {
            for (int i = tid; i < parts; i += kJoinThreads) see(i);
            m = warp_max(m);
            if (lane == 0) max_s[warp] = m;
            __syncthreads();
            m = max_s[lane % kJoinWarps];
        } else {
            for (int i = lane; i < parts; i += 32) see(i);
        }
        m = warp_max(m);
        const int p0 = shared_job ? parts * warp / kJoinWarps : 0;
        const int p1 = shared_job ? parts * (warp + 1) / kJoinWarps : parts;
        float sum;
        float4 acc = join_parts<RT>(a, v0, parts, row, DB * 128, d, p0, p1, m, &sum);
        if (shared_job) {
            acc_s[warp][lane] = acc;
            if (lane == 0) sum_s[warp] = sum;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int i = 1; i < kJoinWarps; ++i) {
                    const float4 o = acc_s[i][lane];
                    acc.x += o.x;
                    acc.y += o.y;
                    acc.z += o.z;
                    acc.w += o.w;
                    sum += sum_s[i];
                }
            }
            __syncthreads();
            if (warp) continue;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        const int rr = it.z + row, tok = rr / a.group, hd = (it.x >> 20) * a.group + rr % a.group;
        uint2 o;
        memcpy(&o.x, &lo, 4);
        memcpy(&o.y, &hi, 4);
        *reinterpret_cast<uint2*>(a.out + (size_t)(it.y + tok) * a.out_row + (size_t)hd * (DB * 128) + d + lane * 4) = o;
    }
}

// ---------------------------------------------------------------- host side
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static EncodeTiled fn = []() -> EncodeTiled {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// Codes as [n_blocks][heads][tokens][head_dim] bytes, in boxes of one block of
// one head x 128 values with the 128-byte swizzle.
bool encode_codes(CUtensorMap* m, const Cache& c, const uint8_t* base) {
    const EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t D = c.cfg.head_dim, bs = c.cfg.block_tokens;
    const cuuint64_t dims[4] = {D, bs, (cuuint64_t)c.cfg.n_kv_heads, (cuuint64_t)c.cfg.n_blocks};
    const cuuint64_t strides[3] = {D, D * bs, (cuuint64_t)c.block_stride};
    const cuuint32_t box[4] = {128, (cuuint32_t)bs, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename S>
cudaError_t run(const Cache& c, const CUtensorMap& km, const CUtensorMap& vm, Args a, cudaStream_t st) {
    a.switch_units = S::SWITCH;
    const int grid = S::CTAS * c.sm_count;
    static_assert(S::CTAS * smem_bytes<S>() <= 232448 + (S::CTAS - 1) * 1024, "the CTAs of an SM must fit its shared memory");
    const size_t chunks = (size_t)grid * S::ROUNDS;
    if (chunks * 2 * S::RT * S::DB * 128 > c.part_o_floats || chunks * 4 * S::RT > c.part_ml_floats || chunks > c.meta_n ||
        chunks > kMaxChunks)
        return cudaErrorInvalidValue;
    attend_kernel<S><<<grid, S::THREADS, smem_bytes<S>(), st>>>(km, vm, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const cudaError_t j = launch_k(join_kernel<S::DB, S::RT>, dim3((unsigned)(4 * c.sm_count)), dim3(kJoinThreads), 0, st, true, a);
    if (j != cudaSuccess) cudaMemsetAsync(c.d_ctrl, 0, 2 * sizeof(int), st);   // what the join does for the next call
    return j;
}

template <int DB, bool SHARED>
cudaError_t run_rows(int rows, const Cache& c, const CUtensorMap& km, const CUtensorMap& vm, const Args& a, cudaStream_t st) {
    if (rows <= 16) return run<Shape<DB, 16, SHARED>>(c, km, vm, a, st);
    // (128-dim heads run two CTAs per SM, which leaves registers for 32 rows)
    if constexpr (DB > 1)
        if (rows > 32) return run<Shape<DB, 64, SHARED>>(c, km, vm, a, st);
    return run<Shape<DB, 32, SHARED>>(c, km, vm, a, st);
}

template <int DB, int RT, bool SHARED>
cudaError_t set_one() {
    using S = Shape<DB, RT, SHARED>;
    return cudaFuncSetAttribute(attend_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<S>());
}
template <int DB, bool SHARED>
cudaError_t set_rows() {
    cudaError_t e = set_one<DB, 16, SHARED>();
    if (e == cudaSuccess) e = set_one<DB, 32, SHARED>();
    if constexpr (DB > 1)
        if (e == cudaSuccess) e = set_one<DB, 64, SHARED>();
    return e;
}

}  // namespace

cudaError_t set_attend_attrs() {
    cudaError_t e = set_rows<1, false>();
    if (e == cudaSuccess) e = set_rows<1, true>();
    if (e == cudaSuccess) e = set_rows<2, false>();
    if (e == cudaSuccess) e = set_rows<2, true>();
    if (e == cudaSuccess) e = set_rows<4, false>();
    if (e == cudaSuccess) e = set_rows<4, true>();
    return e;
}

namespace {
template <int DB, int RT>
void scratch_of(size_t sm_count, size_t* o_floats, size_t* ml_floats, size_t* meta) {
    using S = Shape<DB, RT, false>;
    const size_t chunks = S::CTAS * sm_count * S::ROUNDS;
    const auto most = [](size_t* v, size_t n) { *v = *v < n ? n : *v; };
    most(o_floats, chunks * 2 * RT * DB * 128);
    most(ml_floats, chunks * 2 * RT * 2);
    most(meta, chunks);
}
template <int DB>
void scratch_of_dim(size_t sm_count, size_t* o_floats, size_t* ml_floats, size_t* meta) {
    scratch_of<DB, 16>(sm_count, o_floats, ml_floats, meta);
    scratch_of<DB, 32>(sm_count, o_floats, ml_floats, meta);
    if (DB > 1) scratch_of<DB, 64>(sm_count, o_floats, ml_floats, meta);
}
}  // namespace

void attend_scratch(int sm_count, int head_dim, size_t* o_floats, size_t* ml_floats, size_t* meta) {
    *o_floats = *ml_floats = *meta = 0;
    if (head_dim == 128) scratch_of_dim<1>(sm_count, o_floats, ml_floats, meta);
    else if (head_dim == 256) scratch_of_dim<2>(sm_count, o_floats, ml_floats, meta);
    else scratch_of_dim<4>(sm_count, o_floats, ml_floats, meta);
}

cudaError_t launch_attend(const Cache& c, const kv8_pool& pool, const int32_t* table, const int32_t* len,
                          const int32_t* cu, int n_req, const uint16_t* q, long long q_row, int n_rows, int n_heads,
                          float scale, int window, uint16_t* out, long long out_row, cudaStream_t st) {
    CUtensorMap km, vm;
    const bool shared = c.cfg.shared_kv;
    if (!encode_codes(&km, c, pool.k_codes) || !encode_codes(&vm, c, shared ? pool.k_codes : pool.v_codes))
        return cudaErrorNotSupported;
    Args a{};
    a.q = q;
    a.out = out;
    a.q_row = q_row;
    a.out_row = out_row;
    a.cu = cu;
    a.len = len;
    a.table = table;
    a.ks = pool.k_scale;
    a.vs = shared ? pool.k_scale : pool.v_scale;
    a.part_o = c.d_part_o;
    a.part_ml = c.d_part_ml;
    a.meta = c.d_meta;
    a.ctrl = c.d_ctrl;
    a.err = c.d_err;
    a.n_req = n_req;
    a.n_rows = n_rows;
    a.kv_heads = c.cfg.n_kv_heads;
    a.group = n_heads / c.cfg.n_kv_heads;
    a.per_group = a.group == 1 ? 0 : ~0ull / (unsigned)a.group + 1;
    a.bs_log2 = c.bs_log2;
    a.n_blocks = c.cfg.n_blocks;
    a.max_blocks = c.cfg.max_blocks;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.window = window < (1 << 30) ? window : 0;            // (a request is at most 2^30 tokens long)
    // rows of an average request's KV head, in the smallest row tile that holds them
    const long long rows = (long long)a.group * ((n_rows + n_req - 1) / n_req);
    const int rt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    switch (c.d_blocks * 2 + shared) {
        case 2: return run_rows<1, false>(rt, c, km, vm, a, st);
        case 3: return run_rows<1, true>(rt, c, km, vm, a, st);
        case 4: return run_rows<2, false>(rt, c, km, vm, a, st);
        case 5: return run_rows<2, true>(rt, c, km, vm, a, st);
        case 8: return run_rows<4, false>(rt, c, km, vm, a, st);
        case 9: return run_rows<4, true>(rt, c, km, vm, a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kv8
}  // namespace srh
