// Router and balancing kernels.
//
// Router ("DeepSeek V3 From Scratch", "In code", route(); "The idea"):
//   s = sigmoid(x . W_gate^T) in fp32, v = s + bias, top-k of v with ties to
//   the lower expert index, weights = s of the chosen experts renormalised to
//   sum to 1 (sum in slot order, IEEE division), plus the per-expert count
//   of assignments.
// Bias update ("In code", update_bias(); kbwen.com DeepSeek tag page, "A bias
//   term for each expert"): load = count / T, bias += step * sign(target -
//   load), once per step.
//
// This file holds the SIMT router (fp32 inputs, and bf16 for any shape) and
// the bias update; the top-k / weight / histogram epilogue is shared with
// the tensor-core router (router_tc.cu) through topk.cuh.
#include "common.cuh"
#include "kernels.h"
#include "topk.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// SIMT router.  One CTA = 32 tokens x all E experts, 256 threads.
//  phase 1: thread e accumulates x[t] . W_gate[e] for the CTA's 32 tokens
//           over 32-wide K chunks staged in shared memory (fp32 FFMA).
//  phase 2: sigmoid, scores to shared memory (and to affinity_out).
//  phase 3: warp 0, one thread per token: top-k + weights + histogram.
constexpr int kRtTok = 32;
constexpr int kRtKc = 32;

template <typename Tin, int KMAX>
__global__ void __launch_bounds__(256) router_simt_kernel(const Tin* __restrict__ x, const Tin* __restrict__ wg,
                                                          const float* __restrict__ bias, int T, int d, int E, int k,
                                                          int32_t* __restrict__ idx, float* __restrict__ w,
                                                          int32_t* __restrict__ counts, float* __restrict__ aff,
                                                          int* status) {
    extern __shared__ float sm[];
    const int sstride = E | 1;  // odd row stride: conflict-free column reads
    float* xs = sm;                              // [kRtTok][kRtKc + 1]
    float* ws = xs + kRtTok * (kRtKc + 1);       // [E][kRtKc + 1]
    float* S = ws + E * (kRtKc + 1);             // [kRtTok][sstride]
    float* bs = S + kRtTok * sstride;            // [E]
    int* hist = reinterpret_cast<int*>(bs + E);  // [E]

    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * kRtTok;
    for (int e = tid; e < E; e += blockDim.x) {
        hist[e] = 0;
        bs[e] = bias[e];
    }

    float acc[kRtTok];
#pragma unroll
    for (int t = 0; t < kRtTok; ++t) acc[t] = 0.f;

    for (int c0 = 0; c0 < d; c0 += kRtKc) {
        __syncthreads();
        for (int q = tid; q < kRtTok * kRtKc; q += blockDim.x) {
            const int r = q / kRtKc, c = q % kRtKc;
            const int t = t0 + r;
            xs[r * (kRtKc + 1) + c] = (t < T && c0 + c < d) ? to_f32(x[(size_t)t * d + c0 + c]) : 0.f;
        }
        for (int q = tid; q < E * kRtKc; q += blockDim.x) {
            const int r = q / kRtKc, c = q % kRtKc;
            ws[r * (kRtKc + 1) + c] = (c0 + c < d) ? to_f32(wg[(size_t)r * d + c0 + c]) : 0.f;
        }
        __syncthreads();
        if (tid < E) {
            const float* wr = ws + tid * (kRtKc + 1);
#pragma unroll 4
            for (int c = 0; c < kRtKc; ++c) {
                const float wv = wr[c];
#pragma unroll
                for (int t = 0; t < kRtTok; ++t) acc[t] = fmaf(xs[t * (kRtKc + 1) + c], wv, acc[t]);
            }
        }
    }
    if (tid < E) {
#pragma unroll
        for (int t = 0; t < kRtTok; ++t) {
            const float s = sigmoid_f32(acc[t]);
            S[t * sstride + tid] = s;
            if (aff && t0 + t < T) aff[(size_t)(t0 + t) * E + tid] = s;
        }
    }
    __syncthreads();
    if (tid < kRtTok && t0 + tid < T) {
        const int t = t0 + tid;
        TopK<KMAX> tk;
        tk.init();
        const float* Sr = S + tid * sstride;
        for (int e = 0; e < E; ++e) {
            const float s = Sr[e];
            tk.push(__fadd_rn(s, bs[e]), s, e);
        }
        emit_route<KMAX>(tk, k, idx + (size_t)t * k, w + (size_t)t * k, hist, status);
    }
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x)
        if (hist[e]) atomicAdd(&counts[e], hist[e]);
}

size_t router_simt_smem(int E) {
    const int sstride = E | 1;
    return sizeof(float) * ((size_t)kRtTok * (kRtKc + 1) + (size_t)E * (kRtKc + 1) + (size_t)kRtTok * sstride + E) +
           sizeof(int) * (size_t)E;
}

template <typename Tin, int KMAX>
static cudaError_t launch_router_simt_t(const void* x, const void* wg, const float* bias, int T, int d, int E, int k,
                                        int32_t* idx, float* w, int32_t* counts, float* aff, int* status,
                                        cudaStream_t st) {
    const size_t smem = router_simt_smem(E);
    auto kern = router_simt_kernel<Tin, KMAX>;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    const int grid = (T + kRtTok - 1) / kRtTok;
    kern<<<grid, 256, smem, st>>>(static_cast<const Tin*>(x), static_cast<const Tin*>(wg), bias, T, d, E, k, idx,
                                  w, counts, aff, status);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_router_simt(const void* x, const void* wg, const float* bias, int T, int d, int E, int k,
                               bool bf16, int32_t* idx, float* w, int32_t* counts, float* aff, int* status,
                               cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    if (bf16) {
        return k <= 8 ? launch_router_simt_t<__nv_bfloat16, 8>(x, wg, bias, T, d, E, k, idx, w, counts, aff, status, st)
                      : launch_router_simt_t<__nv_bfloat16, 16>(x, wg, bias, T, d, E, k, idx, w, counts, aff, status,
                                                                 st);
    }
    return k <= 8 ? launch_router_simt_t<float, 8>(x, wg, bias, T, d, E, k, idx, w, counts, aff, status, st)
                  : launch_router_simt_t<float, 16>(x, wg, bias, T, d, E, k, idx, w, counts, aff, status, st);
}

// ---------------------------------------------------------------------------
// Gate logits of an fp32 layer: z = x W_gate^T, FFMA in k order.  A CTA takes
// 32 tokens x 32 experts (small layers: many small tiles fill more SMs than
// the router's 32 tokens x E), each of its 128 threads 2 x 4 of them; 32-wide
// K chunks go through shared memory.  Bound by the latency of a chunk's loads and
// barriers, 1 to 2 us with nothing in flight meanwhile: 17.5 us at d = 512 (64 x 64
// as 512 x 256), 134 at 4096 x 2048 x 64, where FFMA alone would take 15 and the
// library's product takes 62.  fp32 layers are the small ones.
__global__ void __launch_bounds__(128) gate_logits_simt_kernel(const float* __restrict__ x,
                                                               const float* __restrict__ wg, int T, int d, int E,
                                                               float* __restrict__ z) {
    constexpr int KC = 32;
    __shared__ float xs[KC][33], ws[KC][36];
    const int tid = threadIdx.x, t0 = blockIdx.x * 32, e0 = blockIdx.y * 32;
    const int tr = tid >> 3, ec = (tid & 7) * 4;  // tokens tr, tr + 16; experts ec .. ec + 3
    float acc[2][4] = {};
    for (int c0 = 0; c0 < d; c0 += KC) {
        __syncthreads();
        for (int i = tid; i < 32 * KC; i += 128) {
            const int r = i >> 5, c = i & 31;
            const bool in = c0 + c < d;
            xs[c][r] = in && t0 + r < T ? x[(size_t)(t0 + r) * d + c0 + c] : 0.0f;
            ws[c][r] = in && e0 + r < E ? wg[(size_t)(e0 + r) * d + c0 + c] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const float a0 = xs[c][tr], a1 = xs[c][tr + 16];
            const float4 b = *reinterpret_cast<const float4*>(&ws[c][ec]);
            const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[0][i] = fmaf(a0, bv[i], acc[0][i]);
                acc[1][i] = fmaf(a1, bv[i], acc[1][i]);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + tr + 16 * h, e = e0 + ec + i;
            if (t < T && e < E) z[(size_t)t * E + e] = acc[h][i];
        }
}

cudaError_t launch_gate_logits_simt(const float* x, const float* wg, int T, int d, int E, float* logits,
                                    cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const dim3 grid((unsigned)((T + 31) / 32), (unsigned)((E + 31) / 32));
    gate_logits_simt_kernel<<<grid, 128, 0, st>>>(x, wg, T, d, E, logits);
    note_launches(1);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Bias update: one thread per expert, every operation a single IEEE fp32
// rounding (no contraction), so the result is a deterministic function of
// (counts, bias).
__global__ void bias_update_kernel(const int32_t* __restrict__ counts, int T, int E, int k, float step,
                                   const float* __restrict__ target, float* __restrict__ bias,
                                   float* __restrict__ load_out) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= E) return;
    const float load = __fdiv_rn((float)counts[i], (float)T);
    const float tgt = target ? target[i] : __fdiv_rn((float)k, (float)E);
    const float diff = __fsub_rn(tgt, load);
    const float sgn = diff > 0.f ? 1.f : (diff < 0.f ? -1.f : 0.f);
    bias[i] = __fadd_rn(bias[i], __fmul_rn(sgn, step));
    if (load_out) load_out[i] = load;
}

cudaError_t launch_bias_update(const int32_t* counts, int T, int E, int k, float step, const float* target,
                               float* bias, float* load_out, cudaStream_t st) {
    bias_update_kernel<<<(E + 255) / 256, 256, 0, st>>>(counts, T, E, k, step, target, bias, load_out);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
