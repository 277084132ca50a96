// SwiGLU backward from pre-activations saved in 8 bits ("DeepSeek V3 From
// Scratch", "The idea": FP8 with fine-grained quantization tiles; "Scaling
// Efficiency: A Deep Dive into the DeepSeek-V3 Architecture", DeepSeekMoE
// sketch: SwiGLU experts).  gemm_tc.cu's gate/up epilogue writes the codes.
//
// Row r of an expert set, a and g the values of its codes, s = sigmoid(a):
//   h = a s g,  dh = wt u,  da = dh g s (1 + a (1 - s)),  dg = dh a s,
//   routed: dw[q] = sum_i u_i h_i  (h unrounded), wt = w[q], q = perm[r].
//
// HBM bound: per element 2 codes + 2/32 scale bytes and 4 of u in, 4 of dadg
// and 2 of h out, 1.62 GB for 65536 rows of 2048.  245 us in a short run, 254 to
// 264 for calls on end (6.1 to 6.6 TB/s, the rate of a plain copy).  That takes
// four chunks of a row in flight per lane, streaming loads and stores, 4 warps per
// CTA and the hardware's exponential; against the same kernel in one run 8 warps
// took 4 us more, two chunks 10, plain loads and stores 5, one chunk 15, expf 8.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "pdl.h"

namespace moe {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// 2^(b - 127) for a scale byte b <= 254
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// eight E4M3 codes times the tile's scale
__device__ __forceinline__ void decode8(uint2 c, float sc, float (&v)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * i] = f.x * sc;
        v[2 * i + 1] = f.y * sc;
    }
}

// One lane's eight columns of a row: the operands, and what becomes of them.
struct Chunk {
    uint2 ca, cg;
    uint32_t ba, bg;
    float4 u0, u1;
};
__device__ __forceinline__ Chunk load_chunk(const SwigluBwdSaved& p, long long r, const float* u, int c) {
    const size_t o = (size_t)r * p.n + c, so = ((size_t)(c >> 7) * p.rows + r) * 4 + ((c & 127) >> 5);
    Chunk k;
    k.ca = __ldcs(reinterpret_cast<const uint2*>(p.a + o));
    k.cg = __ldcs(reinterpret_cast<const uint2*>(p.g + o));
    k.ba = p.a_scale[so];
    k.bg = p.g_scale[so];
    k.u0 = __ldcs(reinterpret_cast<const float4*>(u + c));
    k.u1 = __ldcs(reinterpret_cast<const float4*>(u + c + 4));
    return k;
}

// One warp per row, eight columns per lane, UNROLL of them in flight.  prow
// (may be null): the row of u, dadg and h; the codes stay at r.
template <int UNROLL>
__global__ void __launch_bounds__(kWarps * 32) swiglu_bwd_saved_kernel(const __grid_constant__ SwigluBwdSaved p) {
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= p.rows) return;  // warp-uniform
    const int n = p.n;
    grid_dependency_wait();
    const long long pr = p.prow ? p.prow[r] : r;
    if (p.prow && (pr < 0 || pr >= p.prow_rows)) {  // warp-uniform
        if (lane == 0) report(p.status, kStDeviceCheck);
        return;
    }
    float wt = 1.0f;
    long long q = r;
    if (p.perm) {
        q = p.perm[r];
        if (q < 0 || q >= p.rows) {
            if (lane == 0) report(p.status, kStDeviceCheck);
            q = -1;
        }
        wt = q < 0 ? 0.0f : p.w[q];
    }
    const float* u = p.u + (size_t)pr * n;
    uint16_t* dadg = p.dadg + (size_t)pr * 2 * n;
    uint16_t* hrow = p.h ? p.h + (size_t)pr * n : nullptr;
    float dot = 0.0f;
    for (int c0 = lane * 8; c0 < n; c0 += 256 * UNROLL) {
        Chunk k[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
            if (c0 + 256 * i < n) k[i] = load_chunk(p, r, u, c0 + 256 * i);
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int c = c0 + 256 * i;
            if (c >= n) break;
            float a[8], g[8];
            decode8(k[i].ca, scale_of(k[i].ba), a);
            decode8(k[i].cg, scale_of(k[i].bg), g);
            const float uv[8] = {k[i].u0.x, k[i].u0.y, k[i].u0.z, k[i].u0.w, k[i].u1.x, k[i].u1.y, k[i].u1.z, k[i].u1.w};
            float da[8], dg[8], h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // s and 1 - s from t = e^-|a|: exact to the ends of the range (t may be subnormal, 1 + t is in
                // [1, 2]).  The hardware's exponential is off by |a| + 4 units of 2^-24, far below bf16's rounding,
                // and dw sums n of them.
                float t, y;
                asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(fabsf(a[j]) * -1.4426950408889634f));
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + t));
                const float ty = t * y;
                const float s = a[j] >= 0.0f ? y : ty, s1 = a[j] >= 0.0f ? ty : y;
                const float as = a[j] * s;
                h[j] = as * g[j];
                dot = fmaf(uv[j], h[j], dot);
                const float dh = wt * uv[j];
                da[j] = dh * g[j] * fmaf(as, s1, s);  // g s (1 + a (1 - s))
                dg[j] = dh * as;
            }
            if (q < 0)  // a row without an assignment: no gradient, whatever its codes and u hold (h is theirs alone)
#pragma unroll
                for (int j = 0; j < 8; ++j) da[j] = dg[j] = 0.0f;
            __stcs(reinterpret_cast<uint4*>(dadg + c),
                   make_uint4(pack2(da[0], da[1]), pack2(da[2], da[3]), pack2(da[4], da[5]), pack2(da[6], da[7])));
            __stcs(reinterpret_cast<uint4*>(dadg + n + c),
                   make_uint4(pack2(dg[0], dg[1]), pack2(dg[2], dg[3]), pack2(dg[4], dg[5]), pack2(dg[6], dg[7])));
            if (hrow)
                __stcs(reinterpret_cast<uint4*>(hrow + c),
                       make_uint4(pack2(h[0], h[1]), pack2(h[2], h[3]), pack2(h[4], h[5]), pack2(h[6], h[7])));
        }
    }
    if (p.perm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0 && q >= 0) p.dw[q] = dot;
    }
}

}  // namespace

cudaError_t launch_swiglu_bwd_saved(const SwigluBwdSaved& p, cudaStream_t st) {
    if (p.rows <= 0) return cudaSuccess;
    const long long blocks = (p.rows + kWarps - 1) / kWarps;
    note_launches(1);
    return launch_after(swiglu_bwd_saved_kernel<4>, dim3((unsigned)blocks), kWarps * 32, 0, 1, st, p);
}

}  // namespace moe
