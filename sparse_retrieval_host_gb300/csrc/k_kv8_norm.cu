// RMS norm of every query and key head with the position rotation in the same
// pass (kv8_norm_rope).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then for each rotated pair (a, b)
//   a' = a cos t - b sin t,  b' = a sin t + b cos t,  t = pos * f_i.
//
// One read and one write of each value: HBM-bound for many tokens, latency for
// a few. A head is held by a group of 8, 16 or 32 lanes, 8 values (one 16-byte
// load) per lane and vector; the sum of squares is a shuffle tree. In the
// HALVES style a value's partner lies rot_dim / 2 further on, in another lane:
// that vector is loaded a second time (from L1) at the same moment as the
// first, which needs no exchange between lanes and no case for odd widths.
//
// The angle: t / 2 pi modulo 1 is all that matters. f_i / 2 pi is held as a
// 64-bit fraction of a turn, so pos * f_i wraps by itself in integer arithmetic
// and keeps 2^-64 * pos of a turn; fp32 would lose 0.06 rad at position 10^6.
// cos and sin of a token are computed once per CTA and shared by its heads.
#include <cuda_bf16.h>

#include "kv8_internal.cuh"

namespace srh {
namespace kv8 {
namespace {

constexpr int kThreads = 256;

struct Args {
    kv8_heads part[2];
    const int32_t* pos;
    const double* inv_freq;
    uint32_t* err;
    int n_tok;
    int vecs;          // head_dim / 8
    float inv_dim;
    int rot_off, rot_dim;
    int pairs;         // style
    float eps;
    int heads_per_cta;
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

// LPH lanes per head, VPL vectors of 8 values per lane, HPG heads of a group at
// a time: their loads are all issued before the first is used, the first ones
// before the token's angles are computed.
template <int LPH, int VPL, int HPG>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ Args a) {
    __shared__ float2 cs[256];          // (cos, sin) of this token's pairs
    const int tid = threadIdx.x;
    const int t = blockIdx.x;
    const int half = a.rot_dim >> 1;
    const int lane = tid % LPH, group = tid / LPH;
    constexpr int kGroups = kThreads / LPH;
    const int total = a.part[0].n_heads + a.part[1].n_heads;
    const int h0 = blockIdx.y * a.heads_per_cta;
    const int h1 = min(total, h0 + a.heads_per_cta);
    uint4 own[HPG][VPL];
    // heads base + i * kGroups of this group; a head past the end loads nothing
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < HPG; ++i) {
            const int g = base + i * kGroups;
            const bool is_k = g >= a.part[0].n_heads;
            const uint16_t* x = (is_k ? a.part[1].x + (size_t)t * a.part[1].x_row : a.part[0].x + (size_t)t * a.part[0].x_row) +
                                (size_t)(is_k ? g - a.part[0].n_heads : g) * a.vecs * 8;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int v = lane + j * LPH;
                own[i][j] = g < h1 && v < a.vecs ? *reinterpret_cast<const uint4*>(x + v * 8) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    load(h0 + group);
    if (tid < half) {
        double turn = a.inv_freq[tid] * 0.15915494309189533576888;   // 1 / (2 pi)
        turn -= floor(turn);
        const unsigned long long step = (unsigned long long)(turn * 18446744073709551616.0);
        const unsigned long long at = (unsigned long long)(long long)a.pos[t] * step;
        // the top 32 bits as a signed fraction of a turn, in units of half a turn
        float s, c;
        sincospif((float)(int)(uint32_t)(at >> 32) * 4.656612873077392578125e-10f, &s, &c);
        cs[tid] = make_float2(c, s);
    }
    __syncthreads();
    for (int first = h0; first < h1; first += kGroups * HPG) {
        if (first > h0) load(first + group);
#pragma unroll
        for (int i = 0; i < HPG; ++i) {
            // every group of a warp goes through the shuffles; those without a head store nothing
            const int g = first + group + i * kGroups;
            if (first + i * kGroups >= h1) break;               // the same for the whole CTA
            const bool is_k = g >= a.part[0].n_heads;
            const kv8_heads& p = a.part[is_k ? 1 : 0];
            const int h = is_k ? g - a.part[0].n_heads : g;
            bool keep = g < h1;
            long long row = t;
            if (keep && p.slot) {
                row = p.slot[t];
                if (row < 0) keep = false;
                else if (row >= p.n_slots) {
                    keep = false;
                    if (lane == 0) atomicOr(a.err, kErrBounds);
                }
            }
            const uint16_t* x = p.x + (size_t)t * p.x_row + (size_t)h * a.vecs * 8;
            uint4 other[VPL];
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int v = lane + j * LPH, e = v * 8 - a.rot_off;
                other[j] = make_uint4(0, 0, 0, 0);
                if (keep && !a.pairs && v < a.vecs && e >= 0 && e < a.rot_dim)
                    other[j] = *reinterpret_cast<const uint4*>(x + v * 8 + (e < half ? half : -half));
                float f[8];
                unpack(own[i][j], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) ss = fmaf(f[q], f[q], ss);
            }
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            __syncwarp();               // in place: every load of this head before any store to it
            const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
            if (!keep) continue;
            uint16_t* out = p.out + (size_t)row * p.out_row + (size_t)h * a.vecs * 8;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int v = lane + j * LPH, e = v * 8 - a.rot_off;
                if (v >= a.vecs) continue;
                float f[8], w[8];
                unpack(own[i][j], f);
                load_w(p.weight, v * 8, w);
#pragma unroll
                for (int q = 0; q < 8; ++q) f[q] *= r * w[q];
                if (e >= 0 && e < a.rot_dim) {
                    if (a.pairs) {
#pragma unroll
                        for (int q = 0; q < 8; q += 2) {
                            const float2 k = cs[(e + q) >> 1];
                            const float u = f[q], z = f[q + 1];
                            f[q] = u * k.x - z * k.y;
                            f[q + 1] = u * k.y + z * k.x;
                        }
                    } else {
                        const bool low = e < half;
                        const int eo = low ? e : e - half;
                        float z[8];
                        unpack(other[j], z);
                        load_w(p.weight, v * 8 + (low ? half : -half), w);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float2 k = cs[eo + q];
                            const float y = z[q] * (r * w[q]);
                            f[q] = low ? f[q] * k.x - y * k.y : y * k.y + f[q] * k.x;
                        }
                    }
                }
                *reinterpret_cast<uint4*>(out + v * 8) =
                    make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
            }
        }
    }
}

}  // namespace

cudaError_t launch_norm_rope(const Cache& c, const kv8_heads& q, const kv8_heads& k, int n_tok, int head_dim,
                             const int32_t* pos, const double* inv_freq, int rot_dim, int rot_off, int style,
                             float eps, cudaStream_t st) {
    Args a{};
    a.part[0] = q;
    a.part[1] = k;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.err = c.d_err;
    a.n_tok = n_tok;
    a.vecs = head_dim / 8;
    a.inv_dim = 1.0f / (float)head_dim;
    a.rot_off = rot_off;
    a.rot_dim = rot_dim;
    a.pairs = style == KV8_ROPE_PAIRS;
    a.eps = eps;
    const int lph = a.vecs <= 8 ? 8 : a.vecs <= 16 ? 16 : 32;
    const int groups = kThreads / lph;
    // a CTA takes a token's heads; while that leaves SMs short of CTAs the heads
    // are split (each CTA computes the token's angles again, a few hundred cycles)
    const int heads = q.n_heads + k.n_heads;
    int per = heads;
    while (per > groups && (long long)n_tok * ((heads + per - 1) / per) < 4ll * c.sm_count) per = (per + 1) / 2;
    a.heads_per_cta = per;
    const dim3 grid((unsigned)n_tok, (unsigned)((heads + per - 1) / per));
    if (lph == 8) norm_rope_kernel<8, 1, 4><<<grid, kThreads, 0, st>>>(a);
    else if (lph == 16) norm_rope_kernel<16, 1, 4><<<grid, kThreads, 0, st>>>(a);
    else if (a.vecs <= 32) norm_rope_kernel<32, 1, 4><<<grid, kThreads, 0, st>>>(a);
    else norm_rope_kernel<32, 2, 2><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kv8
}  // namespace srh
