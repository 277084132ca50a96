// Routing from gate logits and its gradient ("DeepSeek V3 From Scratch", "In
// code", route(): scores, biased choice, weights from the unbiased scores;
// "Scaling Efficiency: A Deep Dive into the DeepSeek-V3 Architecture",
// DeepSeekMoE sketch: softmax gating), with sigmoid or softmax scores and the
// choice limited to the best groups of experts.
//
// Forward, one warp per token:
//   s = sigmoid(z) or softmax(z);  v = s + bias in 64 bits;
//   group value = sum of the group's 1 or 2 largest v; the top_groups best
//   groups are kept (ties: lower group); the k largest v of the kept groups
//   in descending order (ties: lower expert);  w = scale s / (sum of the k s).
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;             // warps (tokens in flight) per CTA
constexpr int kSlots = kMaxExperts / 32;  // experts per lane, lane + 32 * j

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ double neg_inf64() { return __longlong_as_double(0xfff0000000000000ll); }

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The share of each lane's chosen logit in the sum over the chosen scores
// (lanes without one: live false).  s = e^min(z,0) / (1 + e^-|z|) (sigmoid) or
// e^z / const (softmax), with the largest exponent taken out of the ratio, so
// that it stands where every score underflows.
__device__ __forceinline__ double chosen_share(double z, bool live, bool softmax) {
    const double x = softmax ? z : fmin(z, 0.0);
    const double m = warp_max(live ? x : neg_inf64());
    double p = live ? (x == m ? 1.0 : exp(x - m)) : 0.0;
    if (!softmax && live) p /= 1.0 + exp(-fabs(z));
    const double tot = warp_sum(p);
    return tot > 0.0 ? p / tot : 0.0;
}

__global__ void __launch_bounds__(kWarps * 32) route_logits_kernel(const float* __restrict__ logits,
                                                                  const float* __restrict__ bias, int T, int E, int k,
                                                                  RouteOpts o, int32_t* __restrict__ idx,
                                                                  float* __restrict__ w, int32_t* __restrict__ counts,
                                                                  int* status) {
    __shared__ double vrow[kWarps][kMaxExperts];
    __shared__ int hist[kMaxExperts];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < E; e += kWarps * 32) hist[e] = 0;
    __syncthreads();
    const int per = E / o.groups;
    for (int t = blockIdx.x * kWarps + warp; t < T; t += gridDim.x * kWarps) {
        double s[kSlots], v[kSlots];
        bool bad = false;
        double m = neg_inf64();
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int e = lane + 32 * j;
            float z = e < E ? logits[(size_t)t * E + e] : neg_inf();
            if (z != z) {
                bad = true;
                z = neg_inf();
            }
            s[j] = (double)z;
            m = fmax(m, s[j]);
        }
        double den = 1.0;
        if (o.softmax) {
            m = warp_max(m);
            double part = 0.0;
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (s[j] != neg_inf64()) part += s[j] == m ? 1.0 : exp(s[j] - m);
            den = warp_sum(part);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int e = lane + 32 * j;
            const double z = s[j];
            v[j] = neg_inf64();
            if (z == neg_inf64()) {
                s[j] = 0.0;
                continue;
            }
            s[j] = o.softmax ? (z == m ? 1.0 : exp(z - m)) / den : 1.0 / (1.0 + exp(-z));
            const double b = bias ? (double)bias[e] : 0.0;
            if (b != b)
                bad = true;
            else
                v[j] = s[j] + b;
        }
        if (o.top_groups < o.groups) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (lane + 32 * j < E) vrow[warp][lane + 32 * j] = v[j];
            __syncwarp();
            double gv = neg_inf64();
            if (lane < o.groups) {
                double a = neg_inf64(), b = neg_inf64();
                for (int i = 0; i < per; ++i) {
                    const double x = vrow[warp][lane * per + i];
                    if (x > a) {
                        b = a;
                        a = x;
                    } else if (x > b) {
                        b = x;
                    }
                }
                gv = o.group_top == 2 && b != neg_inf64() ? a + b : a;
            }
            int ahead = 0;
            for (int g = 0; g < o.groups; ++g) {
                const double x = __shfl_sync(kFull, gv, g);
                ahead += x > gv || (x == gv && g < lane);
            }
            const unsigned kept = __ballot_sync(kFull, lane < o.groups && ahead < o.top_groups);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (!((kept >> ((lane + 32 * j) / per & 31)) & 1u)) v[j] = neg_inf64();
        }
        // k rounds: the best (largest v, then lowest expert) leaves
        double my_s = 0.0;
        int my_e = -1;
        for (int r = 0; r < k; ++r) {
            double bv = neg_inf64(), bs = 0.0;
            int be = 0x7fffffff;
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (v[j] > bv) {
                    bv = v[j];
                    bs = s[j];
                    be = lane + 32 * j;
                }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const double ov = __shfl_xor_sync(kFull, bv, d), os = __shfl_xor_sync(kFull, bs, d);
                const int oe = __shfl_xor_sync(kFull, be, d);
                if (ov > bv || (ov == bv && oe < be)) {
                    bv = ov;
                    bs = os;
                    be = oe;
                }
            }
            if (bv == neg_inf64()) {
                bad = true;
                break;
            }
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (lane + 32 * j == be) v[j] = neg_inf64();
            if (lane == r) {
                my_s = bs;
                my_e = be;
            }
        }
        if (o.renormalize)
            my_s = chosen_share(my_e >= 0 ? (double)logits[(size_t)t * E + my_e] : 0.0, my_e >= 0, o.softmax);
        if (lane < k) {
            idx[(size_t)t * k + lane] = my_e;
            w[(size_t)t * k + lane] = (float)(my_s * (double)o.scale);
            if (my_e >= 0) atomicAdd(&hist[my_e], 1);
        }
        if (bad) report(status, kStDeviceCheck);
    }
    __syncthreads();
    for (int e = tid; e < E; e += kWarps * 32)
        if (hist[e]) atomicAdd(&counts[e], hist[e]);
}

// Backward, one warp per token: ds from the chosen weights (and dscores),
// through the Jacobian of the scores.
__global__ void __launch_bounds__(kWarps * 32) route_logits_bwd_kernel(const float* __restrict__ logits,
                                                                      const int32_t* __restrict__ idx,
                                                                      const float* __restrict__ dw,
                                                                      const float* __restrict__ dscores, int T, int E,
                                                                      int k, RouteOpts o, float* __restrict__ dlogits,
                                                                      int* status) {
    __shared__ double add[kWarps][kMaxExperts];  // what the chosen slots add: to dz, or to ds (softmax as scored)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= T) return;  // warp-uniform
    double z[kSlots], m = neg_inf64();
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
        const int e = lane + 32 * j;
        const float x = e < E ? logits[(size_t)t * E + e] : neg_inf();
        z[j] = x != x ? neg_inf64() : (double)x;
        m = fmax(m, z[j]);
        add[warp][e] = 0.0;
    }
    m = warp_max(m);
    // chosen slots
    int e = -1;
    double G = 0.0, ze = neg_inf64();
    if (lane < k) {
        e = idx[(size_t)t * k + lane];
        if (e < -1 || e >= E) report(status, kStDeviceCheck);
        if (e < 0 || e >= E) {
            e = -1;
        } else {
            G = (double)dw[(size_t)t * k + lane] * (double)o.scale;
            const float x = logits[(size_t)t * E + e];
            ze = x != x ? neg_inf64() : (double)x;
        }
    }
    double sj = 0.0, part = 0.0;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
        if (z[j] != neg_inf64()) part += z[j] == m ? 1.0 : exp(z[j] - m);
    const double den = warp_sum(part);
    const bool live = e >= 0 && ze != neg_inf64();
    if (live) sj = o.softmax ? (ze == m ? 1.0 : exp(ze - m)) / den : 1.0 / (1.0 + exp(-ze));
    double c = G * sj;  // softmax, as scored: ds; sigmoid: before (1 - s)
    if (o.renormalize) {
        const double p = chosen_share(ze, live, o.softmax);
        const double dot = warp_sum(live ? G * p : 0.0);
        c = live ? p * (G - dot) : 0.0;
    } else if (o.softmax) {
        c = live ? G : 0.0;
    } else {
        c = live ? c : 0.0;
    }
    if (!o.softmax && live) c *= 1.0 / (1.0 + exp(ze));
    __syncwarp();
    for (int r = 0; r < k; ++r) {  // in slot order: an expert listed twice gets the sum
        if (lane == r && live) add[warp][e] += c;
        __syncwarp();
    }
    double dot = 0.0, ds[kSlots];
    if (o.softmax) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int i = lane + 32 * j;
            ds[j] = 0.0;
            if (i < E && z[j] != neg_inf64()) {
                if (dscores) ds[j] += (double)dscores[(size_t)t * E + i];
                if (!o.renormalize) ds[j] += add[warp][i];
                dot += ds[j] * ((z[j] == m ? 1.0 : exp(z[j] - m)) / den);
            }
        }
        dot = warp_sum(dot);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
        const int i = lane + 32 * j;
        if (i >= E) continue;
        double dz = 0.0;
        if (z[j] != neg_inf64()) {
            if (o.softmax) {
                dz = ((z[j] == m ? 1.0 : exp(z[j] - m)) / den) * (ds[j] - dot);
                if (o.renormalize) dz += add[warp][i];
            } else {
                const double s = 1.0 / (1.0 + exp(-z[j]));
                if (dscores) dz = (double)dscores[(size_t)t * E + i] * s * (1.0 / (1.0 + exp(z[j])));
                dz += add[warp][i];
            }
        }
        dlogits[(size_t)t * E + i] = (float)dz;
    }
}

}  // namespace

cudaError_t launch_route_logits(const float* logits, const float* bias, int T, int E, int k, const RouteOpts& o,
                                int32_t* idx, float* w, int32_t* counts, int* status, int num_sms, cudaStream_t st) {
    cudaError_t err = cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)E, st);
    if (err != cudaSuccess || T == 0) return err;
    const int blocks = (T + kWarps - 1) / kWarps;
    const int grid = blocks < 4 * num_sms ? blocks : 4 * num_sms;
    route_logits_kernel<<<grid, kWarps * 32, 0, st>>>(logits, bias, T, E, k, o, idx, w, counts, status);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_route_logits_bwd(const float* logits, const int32_t* idx, const float* dw, const float* dscores,
                                    int T, int E, int k, const RouteOpts& o, float* dlogits, int* status, int num_sms,
                                    cudaStream_t st) {
    (void)num_sms;
    if (T == 0) return cudaSuccess;
    route_logits_bwd_kernel<<<(T + kWarps - 1) / kWarps, kWarps * 32, 0, st>>>(logits, idx, dw, dscores, T, E, k, o,
                                                                              dlogits, status);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace moe
