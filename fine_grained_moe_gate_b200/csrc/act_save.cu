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
// and 2 of h out.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

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

// One warp per row, eight columns per lane.  prow (may be null): the row of u,
// dadg and h; the codes stay at r.
__global__ void __launch_bounds__(kWarps * 32) swiglu_bwd_saved_kernel(SwigluBwdSaved p) {
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (r >= p.rows) return;  // warp-uniform
    const long long pr = p.prow ? p.prow[r] : r;
    float wt = 1.0f;
    long long q = r;
    if (p.perm) {
        q = p.perm[r];
        if (q < 0 || q >= p.rows) {
            if (lane == 0) report(p.status, kStDeviceCheck);
            q = -1;
            wt = 0.0f;
        } else {
            wt = p.w[q];
        }
    }
    const int n = p.n;
    float dot = 0.0f;
    for (int c = lane * 8; c < n; c += 256) {
        const size_t o = (size_t)r * n + c, po = (size_t)pr * n + c;
        const size_t so = ((size_t)(c >> 7) * p.rows + r) * 4 + ((c & 127) >> 5);
        float a[8], g[8];
        decode8(*reinterpret_cast<const uint2*>(p.a + o), scale_of(p.a_scale[so]), a);
        decode8(*reinterpret_cast<const uint2*>(p.g + o), scale_of(p.g_scale[so]), g);
        const float4 u0 = *reinterpret_cast<const float4*>(p.u + po), u1 = *reinterpret_cast<const float4*>(p.u + po + 4);
        const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        float da[8], dg[8], h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = 1.0f / (1.0f + expf(-a[i]));
            const float as = a[i] * s;
            h[i] = as * g[i];
            dot = fmaf(u[i], h[i], dot);
            const float dh = wt * u[i];
            da[i] = q < 0 ? 0.0f : dh * g[i] * s * (1.0f + a[i] * (1.0f - s));
            dg[i] = q < 0 ? 0.0f : dh * as;
        }
        uint4* d0 = reinterpret_cast<uint4*>(p.dadg + (size_t)pr * 2 * n + c);
        uint4* d1 = reinterpret_cast<uint4*>(p.dadg + (size_t)pr * 2 * n + n + c);
        *d0 = make_uint4(pack2(da[0], da[1]), pack2(da[2], da[3]), pack2(da[4], da[5]), pack2(da[6], da[7]));
        *d1 = make_uint4(pack2(dg[0], dg[1]), pack2(dg[2], dg[3]), pack2(dg[4], dg[5]), pack2(dg[6], dg[7]));
        if (p.h)
            *reinterpret_cast<uint4*>(p.h + po) =
                make_uint4(pack2(h[0], h[1]), pack2(h[2], h[3]), pack2(h[4], h[5]), pack2(h[6], h[7]));
    }
    if (p.perm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0 && q >= 0) p.dw[q] = dot;
    }
}

}  // namespace

cudaError_t launch_swiglu_bwd_saved(const SwigluBwdSaved& p, int num_sms, cudaStream_t st) {
    (void)num_sms;
    if (p.rows <= 0) return cudaSuccess;
    const long long blocks = (p.rows + kWarps - 1) / kWarps;
    swiglu_bwd_saved_kernel<<<(unsigned)blocks, kWarps * 32, 0, st>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
