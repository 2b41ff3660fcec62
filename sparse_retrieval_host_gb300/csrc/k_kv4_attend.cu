// Attention over the paged 4-bit cache (kv4_attend), for few query rows per KV head
// (decode steps, drafted tokens of small groups).
//
//   o_r = sum_t w_rt V_t / sum_t w_rt,  w_rt = exp(scale <q_r, K_t>),
//   K_t = km_t + ks_t n_t, V_t = vm_t + vs_t m_t, codes n, m in 0 .. 15
//
// A warp takes 16 tokens at a time (two such steps together for 128-dim heads), and their codes go from memory into the fragments of
// mma.sync m16n8k16 (fp16) without a detour: tokens are the M dimension of S^T = n q^T, head
// dims that of O^T = m^T p. (tcgen05 wants its operands unpacked in shared memory, whose
// bandwidth, not HBM's, would bound a call of few rows: the products of 8 rows are a
// sixth of what these instructions can do.)
//
// Codes need no conversion: a code in the low bits of an fp16 is the subnormal n 2^-24, and
// tensor cores take subnormals as they are. (w & 0x000f000f) is thus two operands for one
// instruction; (w & 0x00f000f0) is two more, 16 times as large, which the queries make up for
// in the first product (dims 1, 3, 5, 7 of each 8 enter 16 times smaller) and the outputs' scale
// in the second. Which dims meet in a k step does not matter as long as both operands agree.
//
// Scores: ks_t <q, n_t> + km_t sum(q), in fp32. Weights carry V's scale in the exponent,
// u = s + log2 vs, p = 2^(u - ref) in fp16, and the minimum enters around the middle of the codes,
//   O = sum p (m - 8) + sum (p / vs) (vm + 8 vs),
// the second sum and the softmax's in fp32 by the threads: what p's rounding does to a token is
// then relative to V's distance from the middle of its range (around vm it would be relative to
// the whole range, and the same for all tokens where all weigh the same). The -8 is taken off by
// sum p, of the rounded p, a row of ones in the second product.
//
// Work: see kv4_split.cuh; a CTA's warps take 16 tokens (32) in turn of a unit's 128, each with references
// and sums of its own, and add up at the end of a segment.
//
// Measured: 64 requests of up to 16,384 tokens, 32 / 8 heads of 128: 138 us, 0.72 of the copy rate over the codes' bytes. The
// arithmetic without loads takes 130 (some 285 instructions per 16 tokens of a warp, ALU 48 % busy, tensor pipe 24 %), loads alone 113
// to 134: both have to overlap almost wholly. Steps of 32 tokens instead of 16 took 174 us to 156, queries in
// shared memory and three CTAs per SM 156 to 142.
#include "kv4_split.cuh"

namespace srh {
namespace kv8 {
namespace {

using namespace split;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kHead = 10.f;            // log2 of the weight that a new reference gives a row's maximum
constexpr float kRoom = 15.5f;           // a row's reference moves when a weight would pass 2^15.5
constexpr float kLeastScale = 5.421010862427522e-20f;   // 2^-64

// DB: head_dim / 128. A row tile has 8 rows (16 took 254 registers, and 2.0 us for 9 to 16 rows against 1.0 of two
// row tiles that read the codes twice, the second time from L2).
template <int DB_>
struct Shape {
    static constexpr int DB = DB_, RT = 8, D = 128 * DB;
    // (with four CTAs 128 registers a thread, which spill: the decode batch 152 us, 142 with three)
    static constexpr int CTAS = DB == 1 ? 3 : 2;
    static constexpr int kPitch = D + 4;                       // floats of a row of the warps' outputs
    static constexpr int kOutBytes = kWarps * RT * kPitch * 4;
    static constexpr int SW = 3;                               // units that stand for a segment's start and end
    static constexpr int kStatBytes = kWarps * RT * 8;         // reference and sum
    // A step of a warp is SUB times 16 tokens: two, so that what a step costs beside its products is
    // shared, where the registers are there.
    static constexpr int SUB = DB == 1 ? 2 : 1;
    static constexpr int kTokens = 16 * SUB, kStride = kWarps * kTokens;     // of a warp's step, of the CTA's
    static constexpr int kCodes = kTokens * D / 2;             // bytes of K or V in a step
    static constexpr int kStage = 2 * kCodes + 8 * kTokens;    // and their scales
    static constexpr int STAGES = DB == 1 ? 2 : 4;             // of each warp's ring
    static constexpr int kRing = kWarps * STAGES * kStage;
    // Queries as operands, and factor, sum and position of each row; twice, as the next segment's are
    // made while this one's outputs are.
    static constexpr int kQBytes = DB * 2048, kRowBytes = RT * 16;
    static constexpr int kOffStat = kOutBytes, kOffRing = kOffStat + kStatBytes, kOffQ = kOffRing + kRing;
    static constexpr int kOffRow = kOffQ + 2 * kQBytes, kOffFirst = kOffRow + 2 * kRowBytes;
};

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(r) : "r"(at));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "r"(at));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
    return r;
}
// D += A B: A 16 x 16 (rows by lane / 4), B 16 x 8 (columns by lane / 4), fp16, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The transpose of an 8 x 8 matrix of fp16, two to a lane.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Where 16-byte piece p of token row t lies among the 16 rows of a stage, so that the reads below meet no
// bank twice: of K 8 rows x 4 pieces at a time (128-byte rows: 2 rows x 4), of V rows 2 c
// of four c, 32 bytes each.
template <int DB>
__device__ __forceinline__ uint32_t k_at(uint32_t t, uint32_t p) {
    return DB == 1 ? t * 64 + p * 16 : t * 128 + ((p ^ ((t & 1) << 2)) << 4);
}
template <int DB>
__device__ __forceinline__ uint32_t v_at(uint32_t t, uint32_t p) {
    if (DB == 2) return t * 128 + ((p ^ (((t >> 1) & 3) << 1)) << 4);
    const uint32_t r = (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3);
    return r * 64 + ((p ^ (r & 2)) << 4);
}

// ---------------------------------------------------------------- the kernel
template <typename S>
__global__ void __launch_bounds__(kThreads, S::CTAS) attend4_kernel(const __grid_constant__ Args a) {
    constexpr int DB = S::DB, RT = S::RT, D = S::D, SUB = S::SUB;
    extern __shared__ __align__(16) unsigned char sm[];
    float* const outs = reinterpret_cast<float*>(sm);                       // [warp][row][kPitch]
    float2* const stats = reinterpret_cast<float2*>(sm + S::kOffStat);      // [warp][row]: reference, sum
    int* const first = reinterpret_cast<int*>(sm + S::kOffFirst);   // units before each request
    __shared__ long long warp_sums[33];
    __shared__ int last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

    Chunks ch;
    if (!count<RT, false, S::SW, kThreads>(a, first, warp_sums, &ch)) {
        pdl_wait();
        return;
    }
    const int cta = blockIdx.x, bsz = 1 << a.bs_log2;
    bool bad = false;
    int u = ch.begin(cta);
    const int u1 = ch.begin(cta + 1);

    // -------------------------------------------------------- the warp's ring
    // Step i takes tokens t_of + kStride i ..; the blocks of the next 32 times 16 tokens are held a
    // lane each.
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm + S::kOffRing + warp * (S::STAGES * S::kStage));
    constexpr int P = 4 * DB, kCopies = S::kCodes / 512;      // 16-byte pieces of a row, and of K a lane
    constexpr int kScaleLanes = S::kTokens / 4;
    const uint32_t k_to = k_at<DB>(lane / P, lane % P), v_to = v_at<DB>(lane / P, lane % P);
    const uint32_t* const scale_src = (lane < kScaleLanes ? a.ks : a.vs - S::kTokens) + lane * 4;
    const bool small = SUB == 2 && bsz == 16;                 // a step has two blocks
    const uint8_t* k_src = nullptr;                           // this lane's, at the head's first token
    const long long v_off = a.vc - a.kc;
    const int32_t* table = nullptr;
    int head_tok = 0, t_of = 0, p_last = 0, see_first = 0, steps = 0, ids = -1, ids_next = -1;
    uint32_t absent = 0;                                      // of the last 32 times 16 tokens asked for, a bit each
    auto blocks = [&](int from) -> int {                      // this lane's of 16 tokens, from step ..
        const int t = t_of + (from + lane / SUB) * S::kStride + (lane % SUB) * 16;
        return from + lane / SUB < steps && t <= p_last ? __ldg(table + (t >> a.bs_log2)) : -1;
    };
    auto ask = [&](int i, uint32_t stage) {                   // step i into its stage
        if (i < steps) {
            if ((i & (32 / SUB - 1)) == 0 && i > 0) {
                ids = ids_next;
                ids_next = blocks(i + 32 / SUB);
            }
            const uint32_t to = ring + stage;
            const int at = (t_of + i * S::kStride) & (bsz - 1);
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                if (sub > 0 && !small) break;
                const int j = (i * SUB + sub) & 31;
                const int id = __shfl_sync(0xffffffffu, ids, j);
                const bool there = (uint32_t)id < (uint32_t)a.n_blocks;
                const uint32_t bit = (SUB == 2 && !small ? 3u : 1u) << j;
                absent = there ? absent & ~bit : absent | bit;        // (a block that is none reads as absent)
                if (!there) {
                    const int t = t_of + i * S::kStride + sub * 16;
                    if (!small || (t <= p_last && t + 15 >= see_first)) bad = true;
                    continue;
                }
                const uint8_t* const kp = k_src + ((long long)id * a.block_stride + at * (D / 2));
                const uint8_t* const vp = kp + v_off;
                const uint32_t* const sp = scale_src + (((size_t)id * a.kv_heads << a.bs_log2) + (head_tok + at));
                if (SUB == 2 && small) {
                    // 16 tokens: half of the copies, and of the scales' lanes
#pragma unroll
                    for (int x = 0; x < kCopies / 2; ++x) {
                        copy16(to + k_to + sub * (S::kCodes / 2) + x * 512, kp + x * 512);
                        copy16(to + v_to + S::kCodes + sub * (S::kCodes / 2) + x * 512, vp + x * 512);
                    }
                    if (lane < 2 * kScaleLanes && (lane % kScaleLanes) < 4) copy16(to + 2 * S::kCodes + lane * 16 + sub * 64, sp);
                } else {
#pragma unroll
                    for (int x = 0; x < kCopies; ++x) {
                        copy16(to + k_to + x * 512, kp + x * 512);
                        copy16(to + (DB == 1 ? v_to : v_at<DB>(lane / P + x * (32 / P), lane % P) - x * 512) + S::kCodes + x * 512,
                               vp + x * 512);
                    }
                    if (lane < 2 * kScaleLanes) copy16(to + 2 * S::kCodes + lane * 16, sp);
                }
            }
        }
        copy_commit();
    };
    auto ask_first = [&](const Segment& s) {
        // the steps that some row sees (what none sees may have been given up)
        const int t0 = s.t0 * kTile + warp * S::kTokens, t1 = min((s.t0 + s.n) * kTile - 1, s.p_hi);
        const int gone = s.p_lo - a.window - t0;              // tokens from t0 on that no row sees any more, less one
        const int skip = a.window && gone >= S::kTokens - 1 ? (gone - S::kTokens + 1) / S::kStride + 1 : 0;
        t_of = t0 + skip * S::kStride;
        p_last = s.p_hi;
        see_first = a.window ? s.p_lo - a.window + 1 : 0;
        steps = s.n > 0 && t_of <= t1 ? (t1 - t_of) / S::kStride + 1 : 0;
        head_tok = s.h << a.bs_log2;
        k_src = a.kc + (size_t)head_tok * (D / 2) + lane * 16;
        table = a.table + (size_t)s.b * a.max_blocks;
        ids = blocks(0);
        ids_next = blocks(32 / SUB);
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) ask(i, i * S::kStage);
    };

    // A segment's queries as B fragments: lane (g, c) holds dims 32 c .. of row g, per 8 dims two k steps.
    // One warp makes them.
    auto stage = [&](const Segment& s, int to) {
        if (warp != 0) return;
        const int row = s.row0 + g, tok = by_group(a, row);
        const bool on = g < s.nr;
        const uint16_t* x = a.q + (size_t)(s.q0 + (on ? tok : 0)) * a.q_row +
                            (size_t)(s.h * a.group + (on ? row - tok * a.group : 0)) * D;
        uint4 w[DB][4];
        uint32_t m = 0;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[d][i] = on ? __ldg(reinterpret_cast<const uint4*>(x + d * 128 + c * 32 + i * 8)) : make_uint4(0, 0, 0, 0);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(w[d][i].x & 0x7fff7fffu, w[d][i].y & 0x7fff7fffu),
                                         __vmaxu2(w[d][i].z & 0x7fff7fffu, w[d][i].w & 0x7fff7fffu)));
            }
        m = max(m & 0xffffu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // to a largest magnitude in [2^14, 2^15)
        const int e = min(max((int)(m >> 7) - 127 - 14, -120), 120);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23), inv16 = inv * 0.0625f;
        float sum = 0.f;
        uint4* const q = reinterpret_cast<uint4*>(sm + S::kOffQ + to * S::kQBytes) + lane;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // dims 0 .. 7: pairs (k, k + 4) as the codes of a word lie
                const uint32_t v[4] = {w[d][i].x, w[d][i].y, w[d][i].z, w[d][i].w};
                q[(d * 4 + i) * 32] = make_uint4(half2_bits(bf_lo(v[0]) * inv, bf_lo(v[2]) * inv),
                                                 half2_bits(bf_hi(v[0]) * inv16, bf_hi(v[2]) * inv16),
                                                 half2_bits(bf_lo(v[1]) * inv, bf_lo(v[3]) * inv),
                                                 half2_bits(bf_hi(v[1]) * inv16, bf_hi(v[3]) * inv16));
#pragma unroll
                for (int k = 0; k < 4; ++k) sum += bf_lo(v[k]) * inv + bf_hi(v[k]) * inv;
            }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // a row that is not finite has no result: NaN
        const float f = m >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
        if (c == 0)      // (codes come as n 2^-24)
            reinterpret_cast<float4*>(sm + S::kOffRow + to * S::kRowBytes)[g] =
                make_float4(f * 16777216.f, f * sum, __int_as_float(on ? s.len - s.nq + tok : -1), 0.f);
    };

    Segment s;
    bool more = next_segment<RT, false, S::SW>(a, first, ch, cta, &u, u1, &s);
    if (more) {
        ask_first(s);
        stage(s, 0);
    }
    __syncthreads();
    for (int turn = 0; more; turn ^= 1) {
        const int row0 = s.row0, nr = s.nr, h = s.h, parts = s.parts;
        // of rows 2 c and 2 c + 1: factor, sum, position
        const float4* const row_at = reinterpret_cast<const float4*>(sm + S::kOffRow + turn * S::kRowBytes) + 2 * c;
        const float4 r0 = row_at[0], r1 = row_at[1];
        const u64 qf = pack(r0.x, r1.x), qs = pack(r0.y, r1.y);
        const int pos[2] = {__float_as_int(r0.z), __float_as_int(r1.z)};
        const uint32_t q_at = (uint32_t)__cvta_generic_to_shared(sm + S::kOffQ + turn * S::kQBytes) + lane * 16;

        float o[DB * 8][4], ones[4];
        u64 l2 = 0, mid2 = 0, nref = 0;                       // sums; minus the references
        uint32_t with_ref = 0;                                // rows that have one, or are none, a bit each
#pragma unroll
        for (int i = 0; i < DB * 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) ones[k] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 * c + k >= nr) with_ref |= 1u << k;
        bool wait_ref = __any_sync(0xffffffffu, with_ref != 3u);

        const int n = steps;
        int t0 = t_of;
        uint32_t out_of = 0, into = (S::STAGES - 1) * S::kStage;      // stages that are read and filled next, in bytes
        for (int i = 0; i < n; ++i, t0 += S::kStride) {
            copy_wait<S::STAGES - 2>();
            __syncwarp();                                     // step i is there; step i - 1 has been read
            ask(i + S::STAGES - 1, into);
            const uint32_t st = ring + out_of;
            into = out_of;
            out_of = out_of == (S::STAGES - 1) * S::kStage ? 0 : out_of + S::kStage;
            const uint32_t off = absent >> (i * SUB & 31);    // 16 tokens that are not there, a bit each
            if ((off & ((1u << SUB) - 1)) == (1u << SUB) - 1) continue;
            const bool odd = t0 + S::kTokens - 1 > s.p_lo || (a.window && t0 <= s.p_hi - a.window) || (off & ((1u << SUB) - 1));

            // scores
            float x[SUB][4];
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                uint32_t w0[SUB][4], w1[SUB][4];
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const uint32_t kp = st + u * (S::kCodes / SUB) + k_at<DB>(g, 4 * d + c);
                    const uint4 k0 = lds128(kp), k1 = lds128(kp + 8 * (D / 2));
                    w0[u][0] = k0.x, w0[u][1] = k0.y, w0[u][2] = k0.z, w0[u][3] = k0.w;
                    w1[u][0] = k1.x, w1[u][1] = k1.y, w1[u][2] = k1.z, w1[u][3] = k1.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 q = lds128(q_at + (d * 4 + j) * 512);
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        if (d == 0 && j == 0)
                            mma_first(x[u], w0[u][j] & 0x000f000fu, w1[u][j] & 0x000f000fu, w0[u][j] & 0x00f000f0u,
                                      w1[u][j] & 0x00f000f0u, q.x, q.y);
                        else
                            mma(x[u], w0[u][j] & 0x000f000fu, w1[u][j] & 0x000f000fu, w0[u][j] & 0x00f000f0u,
                                w1[u][j] & 0x00f000f0u, q.x, q.y);
                    }
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        const uint32_t x0 = w0[u][j] >> 8, x1 = w1[u][j] >> 8;
                        mma(x[u], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, q.z, q.w);
                    }
                }
            }
            // exponents with V's scale, relative to the rows' references
            float iv[SUB][2], cm[SUB][2];                     // of tokens g and g + 8
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t at = st + 2 * S::kCodes + (u * 16 + j * 8 + g) * 4;
                    const uint32_t ksm = lds32(at), vsm = lds32(at + 4 * S::kTokens);
                    const float vsc = fmaxf(bf_lo(vsm), kLeastScale), lv = lg2(vsc);
                    iv[u][j] = rcp(vsc);
                    cm[u][j] = fmaf(8.f, vsc, bf_hi(vsm)) * iv[u][j];
                    const u64 ks2 = pack(bf_lo(ksm), bf_lo(ksm)), km2 = pack(bf_hi(ksm), bf_hi(ksm)), lv2 = pack(lv, lv);
                    const u64 b2 = add2(fma2(km2, qs, lv2), nref);
                    unpack(fma2(mul2(pack(x[u][2 * j], x[u][2 * j + 1]), qf), ks2, b2), x[u][2 * j], x[u][2 * j + 1]);
                }
            if (odd) {
                // (what lies behind the request, in no block, or in one that every row's window has passed, may be anything)
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int tt = t0 + u * 16 + g + 8 * j;
                        const bool none = tt >= s.len || tt < see_first || (off >> u & 1);
                        if (none) iv[u][j] = cm[u][j] = 0.f;
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (none || tt > pos[r] || (a.window && tt <= pos[r] - a.window)) x[u][2 * j + r] = -INFINITY;
                    }
            }
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < SUB; ++u) top = fmaxf(fmaxf(top, fmaxf(x[u][0], x[u][1])), fmaxf(x[u][2], x[u][3]));
            if (__any_sync(0xffffffffu, top > kRoom) || wait_ref) {
                // new references: the maximum of the step's tokens per row
                float f[2], nr2[2];
                unpack(nref, nr2[0], nr2[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t bit = 1u << j;
                    float m = -INFINITY;
#pragma unroll
                    for (int u = 0; u < SUB; ++u) m = fmaxf(m, fmaxf(x[u][j], x[u][j + 2]));
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                    f[j] = 1.f;
                    // every row that grew, while at it; a row's first tokens bring it its first one
                    if (m > kHead || (!(with_ref & bit) && m != -INFINITY)) {
                        const float by = kHead - m;
                        f[j] = with_ref & bit ? ex2(by) : 0.f;
                        nr2[j] += by;
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            x[u][j] += by;
                            x[u][j + 2] += by;
                        }
                        with_ref |= bit;
                    }
                }
                const u64 f2 = pack(f[0], f[1]);
                nref = pack(nr2[0], nr2[1]);
                l2 = mul2(l2, f2);
                mid2 = mul2(mid2, f2);
#pragma unroll
                for (int w = 0; w < 4; ++w) ones[w] *= f[w & 1];
#pragma unroll
                for (int m = 0; m < DB * 8; ++m)
#pragma unroll
                    for (int w = 0; w < 4; ++w) o[m][w] *= f[w & 1];
                wait_ref = __any_sync(0xffffffffu, with_ref != 3u);
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t p[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float w0 = ex2(x[u][2 * j]), w1 = ex2(x[u][2 * j + 1]);
                    const u64 w2 = pack(w0, w1);
                    l2 = fma2(w2, pack(iv[u][j], iv[u][j]), l2);
                    mid2 = fma2(w2, pack(cm[u][j], cm[u][j]), mid2);
                    p[j] = transposed(half2_bits(w0, w1));
                }
                constexpr uint32_t one = 0x3c003c00u;
                mma(ones, one, one, one, one, p[0], p[1]);
                // outputs. V: tokens 2 c, 2 c + 1, and 8 more on, dims 16 DB g ..
                uint32_t v[4][2 * DB];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = st + S::kCodes + u * (S::kCodes / SUB) + v_at<DB>(2 * c + (j & 1), DB == 1 ? g >> 1 : g) +
                                        (j >> 1) * (8 * D / 2);
                    if (DB == 1) {
                        const uint2 w = lds64(at + (g & 1) * 8);
                        v[j][0] = w.x;
                        v[j][1] = w.y;
                    } else {
                        const uint4 w = lds128(at);
                        v[j][0] = w.x;
                        v[j][1] = w.y;
                        v[j][2 * DB - 2] = w.z;
                        v[j][2 * DB - 1] = w.w;
                    }
                }
#pragma unroll
                for (int j = 0; j < 2 * DB; ++j) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t x0 = __byte_perm(v[0][j], v[1][j], half ? 0x7632 : 0x5410);
                        uint32_t x1 = __byte_perm(v[2][j], v[3][j], half ? 0x7632 : 0x5410);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            mma(o[j * 4 + half * 2 + m], x0 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x000f000fu,
                                x1 & 0x00f000f0u, p[0], p[1]);
                            x0 >>= 8;
                            x1 >>= 8;
                        }
                    }
                }
            }
        }

        // the next segment's first steps on their way
        Segment then;
        __syncwarp();

        more = next_segment<RT, false, S::SW>(a, first, ch, cta, &u, u1, &then);
        if (more) {
            ask_first(then);
            stage(then, turn ^ 1);
        }

        // -------------------------------------------------------- the warps' sums together
        float l[2], mid[2], nr2[2];
        unpack(l2, l[0], l[1]);
        unpack(mid2, mid[0], mid[1]);
        unpack(nref, nr2[0], nr2[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                l[j] += __shfl_xor_sync(0xffffffffu, l[j], x);
                mid[j] += __shfl_xor_sync(0xffffffffu, mid[j], x);
            }
            const int row = 2 * c + j;
            if (g == 0) stats[warp * RT + row] = make_float2(-nr2[j], l[j]);
            float* dst = outs + (warp * RT + row) * S::kPitch;
#pragma unroll
            for (int m = 0; m < DB * 8; ++m) {
                // o[m][j]: an even dim, n 2^-24; o[m][j + 2]: the next one, 16 times that
                const float add = fmaf(-8.f, ones[j], mid[j]);
                *reinterpret_cast<float2*>(dst + (m * 8 + g) * 2) =
                    make_float2(fmaf(o[m][j], 16777216.f, add), fmaf(o[m][j + 2], 1048576.f, add));
            }
        }
        __syncthreads();
        const size_t slot = slot_of(s.v0, s.part);
        // two dims of a row per thread and turn
        for (int x = tid; x < nr * (D / 2); x += kThreads) {
            const int row = x / (D / 2), d = (x - row * (D / 2)) * 2;
            const int in_g = d % (16 * DB), from = ((in_g >> 1) * 8 + d / (16 * DB)) * 2;
            float m = kLow;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (stats[w * RT + row].y != 0.f) m = fmaxf(m, stats[w * RT + row].x);
            float sum = 0.f;
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 st = stats[w * RT + row];
                if (st.y == 0.f) continue;
                const float f = ex2(st.x - m);
                const float2 v = *reinterpret_cast<const float2*>(outs + (w * RT + row) * S::kPitch + from);
                sum = fmaf(f, st.y, sum);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
            }
            if (parts == 1) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int rr = row0 + row, tok = by_group(a, rr);
                const __nv_bfloat162 v = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
                *reinterpret_cast<__nv_bfloat162*>(a.out + (size_t)(s.q0 + tok) * a.out_row +
                                                   (size_t)(h * a.group + rr - tok * a.group) * D + d) = v;
            } else {
                *reinterpret_cast<float2*>(a.part_o + (slot * RT + row) * D + d) = acc;
                if (d == 0) reinterpret_cast<float2*>(a.part_ml)[slot * RT + row] = make_float2(m, sum);
            }
        }
        if (parts > 1) {
            __syncthreads();
            finish<RT, D>(a, s, tid, kThreads, &last);
        }
        __syncthreads();                                      // the next segment's outputs take this one's place
        s = then;
    }
    copy_wait<0>();
    if (bad) atomicOr(a.err, kErrBounds);
    pdl_wait();                          // this kernel is not over before the one that it runs beside
}

template <typename S>
size_t smem_bytes(int n_req) {
    return S::kOffFirst + (size_t)n_req * sizeof(int);
}

template <typename S>
cudaError_t run(const Cache& c, Args a, bool beside, cudaStream_t st) {
    const int grid = S::CTAS * c.sm_count;
    size_t o = 0, ml = 0, meta = 0;
    chunk4_scratch(c.sm_count, &o, &ml, &meta);
    // (behind what the kernel beside it has)
    a.part_o = c.d_part_o + o;
    a.part_ml = c.d_part_ml + ml;
    a.arrived_n = grid;
    if (o + (size_t)grid * 2 * S::RT * S::D > c.part_o_floats || ml + (size_t)grid * 4 * S::RT > c.part_ml_floats ||
        3 * (size_t)grid > c.arrived_n)
        return cudaErrorInvalidValue;
    return launch_k(attend4_kernel<S>, dim3(grid), dim3(kThreads), smem_bytes<S>(a.n_req), st, beside, a);
}
template <typename S>
cudaError_t set_one() {
    return cudaFuncSetAttribute(attend4_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<S>(kMaxBatch));
}

// Rows per KV head up to which a request goes by this kernel where the other one runs too. A tile of 128 tokens costs an
// SM some 0.5 us per 8 rows here, and 1.2 there for up to 128: 64 requests of up to 16,384 tokens with 16 heads a group take 265 us
// here and 510 there, 8 with 24 heads 73 and 79. Of 256 dims 1.0 per 8 rows against 2.3 (with two lanes that share few
// units more): 24 requests of 8,192 tokens with 32 heads a group 113 us here and 128 there.
constexpr int kFew = 24;
constexpr int kFewWide = 32;
// Rows per KV head of a whole call up to which idle table rows (fewer rows than requests) make no difference. A call of no more rows
// than requests is a decode step as a rule, and launching both kernels costs one 4 us (20 to 140 us long); but it may be a
// prompt whose neighbours have no tokens, which only the device knows. On 16,384 tokens one of 128 rows a KV head takes 66 us
// here and 34 there (on 2,048 22 and 29), of 256 116 and 48, of 4,096 1,586 and 293.
constexpr int kIdle = 128;

}  // namespace

void attend4_scratch(int sm_count, size_t* o_floats, size_t* ml_floats, size_t* meta, size_t* arrivals) {
    chunk4_scratch(sm_count, o_floats, ml_floats, meta);
    *o_floats += (size_t)sm_count * 2 * 2 * 16 * 128;
    *ml_floats += (size_t)sm_count * 2 * 4 * 16;
    *arrivals = (size_t)sm_count * 9;
}

cudaError_t set_attend4_attrs() {
    cudaError_t e = set_one<Shape<1>>();
    if (e == cudaSuccess) e = set_one<Shape<2>>();
    if (e == cudaSuccess) e = set_chunk4_attrs();
    return e;
}

cudaError_t launch_attend4(const Cache& c, const kv4_pool& pool, const int32_t* table, const int32_t* len,
                           const int32_t* cu, int n_req, const uint16_t* q, long long q_row, int n_rows, int n_heads,
                           float scale, int window, uint16_t* out, long long out_row, cudaStream_t st) {
    Args a{};
    a.q = q;
    a.out = out;
    a.q_row = q_row;
    a.out_row = out_row;
    a.block_stride = pool.block_stride;
    a.cu = cu;
    a.len = len;
    a.table = table;
    a.kc = pool.k_codes;
    a.vc = pool.v_codes;
    a.ks = reinterpret_cast<const uint32_t*>(pool.k_scale);
    a.vs = reinterpret_cast<const uint32_t*>(pool.v_scale);
    a.part_o = c.d_part_o;
    a.part_ml = c.d_part_ml;
    a.arrived = c.d_arrived;
    a.meta = c.d_meta;
    a.ctrl = c.d_ctrl;
    a.err = c.d_err;
    a.n_req = n_req;
    a.n_rows = n_rows;
    a.kv_heads = c.cfg.n_kv_heads;
    a.group = n_heads / c.cfg.n_kv_heads;
    a.per_group = a.group == 1 ? 0 : ~0ull / (unsigned)a.group + 1;
    a.rows_lo = 0;
    a.rows_hi = 1 << 30;
    a.bs_log2 = c.bs_log2;
    a.n_blocks = c.cfg.n_blocks;
    a.max_blocks = c.cfg.max_blocks;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.window = window < (1 << 30) ? window : 0;            // (a request is at most 2^30 tokens long)
    const int dim = c.cfg.head_dim, few = dim == 128 ? kFew : kFewWide;
    const long long all = (long long)a.group * n_rows;
    // One token per request, as far as the host can see: this kernel alone. Otherwise requests of more
    // than `few` rows go by the other one, in the same call, as only the device knows which those are.
    const bool idle = n_rows < n_req;
    const bool beside = all > few && (n_rows > n_req || a.group > few || (idle && all > kIdle));
    if (beside) {
        size_t o = 0, ml = 0, meta = 0;
        chunk4_scratch(c.sm_count, &o, &ml, &meta);
        if (o > c.part_o_floats || ml > c.part_ml_floats || meta > c.meta_n) return cudaErrorInvalidValue;
        Args big = a;
        big.rows_lo = a.rows_hi = few;
        const cudaError_t e = launch_chunk4(c.sm_count, dim, big, st);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = cudaSuccess;
    // (with more heads than that a group, none is left for this one; in a decode step the other has nothing to run beside)
    const bool early = beside && !idle;
    if (!beside || a.group <= few) e = dim == 128 ? run<Shape<1>>(c, a, early, st) : run<Shape<2>>(c, a, early, st);
    if (beside && e == cudaSuccess) e = launch_join4(c.sm_count, dim, a, st);
    return e;
}

}  // namespace kv8
}  // namespace srh
