// RMS norm of every query and key head with the position rotation in the same
// pass (kv8_norm_rope; kv8_norm_rope_axes with a position per axis).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then for each rotated pair (a, b)
//   a' = a cos t - b sin t,  b' = a sin t + b cos t,  t = pos * f_i.
//
// One read and one write of each value: HBM-bound for many tokens, latency for
// a few. A warp takes a range of heads, token after token: the ranges are equal
// and as many as the GPU holds warps, so all of them end together and step, the
// table of angles per position, is made once per CTA (shares of single tokens in
// 2.5 waves: 6,143 tokens of 40 heads 31 us, now 28; 700 tokens 10.5, now 7.4).
// 8, 16 or 32 lanes to a head, 8 values (one 16-byte load) per lane and vector.
// A lane holds the same dims of every head, so weight, cos and sin come down to
// two factors per value in registers, made once per token and kind of head:
//   out_i = r (x_i A_i + x_partner(i) B_i).
// (With a CTA per token and 2-3 heads per lane the factors cost more instructions
// than the heads: 35 M against 9 M for 6,143 tokens of 40 heads, 56 us.)
// In the HALVES style a value's partner lies rot_dim / 2 further on, in another
// lane: that vector is loaded a second time (from L1), which needs no exchange
// between lanes and no case for odd widths.
//
// The angle: t / 2 pi modulo 1 is all that matters. f_i / 2 pi is held as a
// 64-bit fraction of a turn, so pos * f_i wraps by itself in integer arithmetic.
// What it loses is pos times the rounding of f_i / 2 pi in fp64 (about 2^-52 of it;
// the fraction's own 2^-64 is less), and 2^-26 of a turn as the fraction becomes
// fp32: 1e-7 rad at position 10^6 with f_i = 1, where an fp32 angle is off by up to
// 0.03.
//
// With several axes a token has up to 8 positions, a lane of its warp each, and a
// pair of dims takes the one of its axis by a shuffle while the angles are made: the
// rest of the kernel does not know of it.
#include <cuda_bf16.h>

#include "kv8_internal.cuh"

namespace srh {
namespace kv8 {
namespace {

constexpr int kThreads = 128;

struct Args {
    kv8_heads part[2];
    const int32_t* pos;
    const double* inv_freq;
    const uint8_t* axis;   // of each pair; NULL: one position per token
    long long pos_row;
    int n_axes;
    uint32_t* err;
    int n_tok;
    int vecs;          // head_dim / 8
    float inv_dim;
    int rot_off, rot_dim;
    int pairs;         // style
    float eps;
    int heads_per_warp;
};

__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
// Pairs of fp32 values in one 64-bit register (one instruction for both).
using u64 = unsigned long long;
__device__ __forceinline__ u64 pair(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(u64 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
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
__device__ __forceinline__ void load_w(const float* w, int e, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 1.f;
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + e)), b = __ldg(reinterpret_cast<const float4*>(w + e + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// LPH lanes per head, VPL vectors of 8 values per lane; a group of lanes loads
// HPG heads before it uses the first.
template <int LPH, int VPL, int HPG, int CTAS, bool AXES>
__global__ void __launch_bounds__(kThreads, CTAS) norm_rope_kernel(const __grid_constant__ Args a) {
    constexpr int kWarps = kThreads / 32, G = 32 / LPH;    // heads of a warp at a time
    __shared__ unsigned long long step[256];               // turns per position, as 64-bit fractions
    __shared__ uint8_t axis[256];
    __shared__ alignas(16) float cosv[kWarps][256], sinv[kWarps][256];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int half = a.rot_dim >> 1;
    for (int i = tid; i < half; i += kThreads) {
        double turn = a.inv_freq[i] * 0.15915494309189533576888;   // 1 / (2 pi)
        turn -= floor(turn);
        step[i] = (unsigned long long)(turn * 18446744073709551616.0);
        if (AXES) {
            int of = a.axis[i];
            if (of >= a.n_axes) {       // no such axis: the pair stays as it is
                if (blockIdx.x == 0) atomicOr(a.err, kErrBounds);
                of = 0;
                step[i] = 0;
            }
            axis[i] = (uint8_t)of;
        }
    }
    __syncthreads();
    const int lane = tid % LPH, group = (tid & 31) / LPH;
    const int heads = a.part[0].n_heads + a.part[1].n_heads;
    bool turned[VPL];                   // this lane's vector lies in the rotated dims
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = (lane + j * LPH) * 8 - a.rot_off;
        turned[j] = e >= 0 && e < a.rot_dim;
    }
    // this warp's heads, of one token after another
    const long long at0 = ((long long)blockIdx.x * kWarps + warp) * a.heads_per_warp;
    const long long at1 = min(at0 + a.heads_per_warp, (long long)a.n_tok * heads);
    if (at0 >= at1) return;             // whole warps
    int t = (int)(at0 / heads), w0 = (int)(at0 - (long long)t * heads);
    int left = (int)(at1 - at0);
    // a token's position (AXES: lane i holds the one of axis i)
    auto position = [&](int of) {
        if (!AXES) return half ? a.pos[of] : 0;
        return half && (tid & 31) < a.n_axes ? a.pos[(tid & 31) * a.pos_row + of] : 0;
    };
    int pos = position(t);
#pragma unroll 1
    for (; left > 0; ++t, w0 = 0) {
        const int w1 = min(heads, w0 + left);
        left -= w1 - w0;
        const int here = pos;
        if (left > 0) pos = position(t + 1);
        __syncwarp();                   // the last token's angles have been read
        for (int i0 = 0; i0 < half; i0 += 32) {
            const int i = i0 + (tid & 31);
            const int mine = AXES ? __shfl_sync(0xffffffffu, here, i < half ? axis[i] : 0) : here;
            if (i >= half) break;
            const unsigned long long at = (unsigned long long)(long long)mine * step[i];
            // the top 32 bits as a signed fraction of a turn, in units of half a turn
            float s, c;
            sincospif((float)(int)(uint32_t)(at >> 32) * 4.656612873077392578125e-10f, &s, &c);
            cosv[warp][i] = c;
            sinv[warp][i] = s;
        }
        __syncwarp();
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
            const kv8_heads& p = a.part[kind];
            const int shift = kind ? a.part[0].n_heads : 0;
            const int h0 = max(0, w0 - shift), h1 = min(p.n_heads, w1 - shift);
            if (h0 >= h1) continue;
            long long row = t;
            if (p.slot) {
                row = p.slot[t];
                if (row < 0) continue;
                if (row >= p.n_slots) {
                    if ((tid & 31) == 0) atomicOr(a.err, kErrBounds);
                    continue;
                }
            }
            const uint16_t* x = p.x + (size_t)t * p.x_row;
            uint16_t* out = p.out + (size_t)row * p.out_row;
            // the factors of this lane's dims
            float A[VPL][8], B[VPL][8];
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int v = lane + j * LPH, e = v * 8 - a.rot_off;
#pragma unroll
                for (int q = 0; q < 8; ++q) A[j][q] = B[j][q] = 0.f;
                if (v >= a.vecs) continue;
                load_w(p.weight, v * 8, A[j]);
                if (!turned[j]) continue;
                if (a.pairs) {
#pragma unroll
                    for (int q = 0; q < 8; q += 2) {
                        const float c = cosv[warp][(e + q) >> 1], s = sinv[warp][(e + q) >> 1];
                        const float u = A[j][q], z = A[j][q + 1];
                        A[j][q] = u * c;
                        B[j][q] = -z * s;
                        A[j][q + 1] = z * c;
                        B[j][q + 1] = u * s;
                    }
                } else {
                    const bool low = e < half;
                    const int eo = low ? e : e - half;
                    load_w(p.weight, v * 8 + (low ? half : -half), B[j]);
#pragma unroll
                    for (int q = 0; q < 8; q += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(&cosv[warp][eo + q]);
                        const float4 s = *reinterpret_cast<const float4*>(&sinv[warp][eo + q]);
                        const float sg = low ? -1.f : 1.f;
                        A[j][q] *= c.x; A[j][q + 1] *= c.y; A[j][q + 2] *= c.z; A[j][q + 3] *= c.w;
                        B[j][q] *= sg * s.x; B[j][q + 1] *= sg * s.y; B[j][q + 2] *= sg * s.z; B[j][q + 3] *= sg * s.w;
                    }
                }
            }
            for (int first = h0; first < h1; first += G * HPG) {
                uint4 own[HPG][VPL];
#pragma unroll
                for (int i = 0; i < HPG; ++i) {
                    const int h = first + group + i * G;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        const int v = lane + j * LPH;
                        own[i][j] = h < h1 && v < a.vecs ? *reinterpret_cast<const uint4*>(x + (size_t)(h * a.vecs + v) * 8)
                                                         : make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < HPG; ++i) {
                    if (first + i * G >= h1) break;            // the same for the whole warp
                    const int h = first + group + i * G;
                    uint4 other[VPL];                          // the partners: in L1 by now
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        const int v = lane + j * LPH;
                        other[j] = make_uint4(0, 0, 0, 0);
                        if (h < h1 && v < a.vecs && !a.pairs && turned[j])
                            other[j] = *reinterpret_cast<const uint4*>(x + (size_t)(h * a.vecs + v) * 8 +
                                                                       (v * 8 - a.rot_off < half ? half : -half));
                    }
                    u64 sq = 0;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        float f[8];
                        unpack(own[i][j], f);
#pragma unroll
                        for (int q = 0; q < 8; q += 2) sq = fma2(pair(f[q], f[q + 1]), pair(f[q], f[q + 1]), sq);
                    }
                    float ss, s1;
                    unpair(sq, ss, s1);
                    ss += s1;
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    __syncwarp();           // in place: every load of this head before any store to it
                    const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        const int v = lane + j * LPH;
                        float f[8], z[8];
                        unpack(own[i][j], f);
                        unpack(other[j], z);                   // zeros where nothing is rotated
                        if (a.pairs && turned[j]) {
#pragma unroll
                            for (int q = 0; q < 8; q += 2) {
                                z[q] = f[q + 1];
                                z[q + 1] = f[q];
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 8; q += 2) {
                            const u64 zb = mul2(pair(z[q], z[q + 1]), pair(B[j][q], B[j][q + 1]));
                            unpair(mul2(fma2(pair(f[q], f[q + 1]), pair(A[j][q], A[j][q + 1]), zb), pair(r, r)), f[q], f[q + 1]);
                        }
                        if (h < h1 && v < a.vecs)
                            *reinterpret_cast<uint4*>(out + (size_t)(h * a.vecs + v) * 8) =
                                make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                    }
                }
            }
        }
    }
}

template <bool AXES>
void launch_kernel(int lph, unsigned grid, const Args& a, cudaStream_t st) {
    if (lph == 8) norm_rope_kernel<8, 1, 3, 8, AXES><<<grid, kThreads, 0, st>>>(a);
    else if (lph == 16) norm_rope_kernel<16, 1, 3, 8, AXES><<<grid, kThreads, 0, st>>>(a);
    else if (a.vecs <= 32) norm_rope_kernel<32, 1, 3, 8, AXES><<<grid, kThreads, 0, st>>>(a);
    else norm_rope_kernel<32, 2, 2, 5, AXES><<<grid, kThreads, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_norm_rope(const Cache& c, const kv8_heads& q, const kv8_heads& k, int n_tok, int head_dim,
                             const int32_t* pos, long long pos_row, int n_axes, const uint8_t* axis,
                             const double* inv_freq, int rot_dim, int rot_off, int style, float eps, cudaStream_t st) {
    Args a{};
    a.part[0] = q;
    a.part[1] = k;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.axis = axis;
    a.pos_row = pos_row;
    a.n_axes = n_axes;
    a.err = c.d_err;
    a.n_tok = n_tok;
    a.vecs = head_dim / 8;
    a.inv_dim = 1.0f / (float)head_dim;
    a.rot_off = rot_off;
    a.rot_dim = rot_dim;
    a.pairs = style == KV8_ROPE_PAIRS;
    a.eps = eps;
    const int lph = a.vecs <= 8 ? 8 : a.vecs <= 16 ? 16 : 32;
    // equal ranges of heads for the warps that the GPU holds (20 a SM with two vectors
    // per lane), of whole loads; each warp makes the angles and factors of its tokens
    const int heads = q.n_heads + k.n_heads, at_once = 32 / lph;
    const long long total = (long long)n_tok * heads, room = (a.vecs <= 32 ? 32ll : 20ll) * c.sm_count;
    long long per = (total + room - 1) / room;
    per = (per + at_once - 1) / at_once * at_once;
    a.heads_per_warp = (int)per;
    const long long warps = (total + per - 1) / per;
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    // CTAs per SM and heads loaded at once: bytes in flight come from warps rather
    // than from loads of one warp (one prompt chunk of 6,143 tokens x 40 heads x 128:
    // 28.0 us with 3, 28.7 with 4, 28.2 with 2, 32 with 1; 6 CTAs with 4 28.2); two
    // vectors a lane need more registers, and a decode step is latency-bound either way
    if (axis) launch_kernel<true>(lph, grid, a, st);
    else launch_kernel<false>(lph, grid, a, st);
    return cudaGetLastError();
}

}  // namespace kv8
}  // namespace srh
