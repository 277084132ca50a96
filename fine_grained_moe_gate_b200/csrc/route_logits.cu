// Routing from gate logits and its gradient ("DeepSeek V3 From Scratch", "In
// code", route(): scores, biased choice, weights from the unbiased scores;
// "Scaling Efficiency: A Deep Dive into the DeepSeek-V3 Architecture",
// DeepSeekMoE sketch: softmax gating), with sigmoid or softmax scores and the
// choice limited to the best groups of experts.
//
// Forward, one warp per token:
//   s = sigmoid(z) or softmax(z);  v = s + bias;
//   group value = sum of the group's 1 or 2 largest v; the top_groups best
//   groups are kept (ties: lower group); the k largest v of the kept groups
//   in descending order (ties: lower expert);  w = scale s / (sum of the k s).
// v is defined in 64 bits.  The kernel forms it in 32 and bounds the error:
// where two values whose order matters are closer than the bound, the values
// concerned are formed again in 64 bits.
//
// Backward, one warp per token, for the choice made:  with G = scale dw,
//   renormalised:  dz_j = p_j (G_j - sum G p) (sigmoid: times 1 - s_j), p the
//     chosen scores' shares, whatever the other experts' logits are;
//   as scored:     ds_j += G_j;
//   dense part:    sigmoid  dz = ds s (1 - s),  softmax  dz = s (ds - sum ds s).
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxK = 16;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ double neg_inf64() { return __longlong_as_double(0xfff0000000000000ll); }

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
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

// VPT consecutive floats of a row of E, from e0 on (elements past the row:
// fill).  vec: E % 4 == 0, the row starts 16-byte aligned.
template <int VPT>
__device__ __forceinline__ void load_row(const float* row, int e0, int E, bool vec, float fill, float (&v)[VPT]) {
    if (VPT % 4 == 0 && vec) {
#pragma unroll
        for (int j = 0; j < VPT; j += 4) {
            float4 x = make_float4(fill, fill, fill, fill);
            if (e0 + j < E) x = *reinterpret_cast<const float4*>(row + e0 + j);
            v[j] = x.x;
            v[j + 1 < VPT ? j + 1 : j] = x.y;
            v[j + 2 < VPT ? j + 2 : j] = x.z;
            v[j + 3 < VPT ? j + 3 : j] = x.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j) v[j] = e0 + j < E ? row[e0 + j] : fill;
    }
}

// A candidate of the choice: its 32-bit value and its expert.
struct Cand {
    float v;
    int e;
};
// Scratch of one warp.
struct alignas(16) WarpMem {
    double d[kMaxExperts];        // 64-bit values, or all experts' 32-bit values
    Cand cand[kMaxExperts + 2];   // in any order
    Cand sorted[kMaxK + 2];       // the k + 1 best, descending
};
static_assert(sizeof(WarpMem) % 16 == 0, "vector reads in every warp's copy");

struct RouteArgs {
    const float* logits;
    const float* bias;
    int T, E, k;
    int per_inv;  // ceil(2^16 / experts of a group): e / per = e per_inv >> 16 for e, per <= 256
    RouteOpts o;
    int32_t* idx;
    float* w;
    int32_t* counts;
    int* status;
};

// ---- 64-bit values, for what the 32-bit ones leave open ----

struct Softmax64 {
    double m, den;
};
__device__ Softmax64 softmax64(const float* row, int E, int lane) {
    double m = neg_inf64();
    for (int e = lane; e < E; e += 32) {
        const float z = row[e];
        if (z == z) m = fmax(m, (double)z);
    }
    m = warp_max(m);
    double part = 0.0;
    for (int e = lane; e < E; e += 32) {
        const double z = (double)row[e];
        if (z == z && z != neg_inf64()) part += z == m ? 1.0 : exp(z - m);
    }
    return {m, warp_sum(part)};
}
// v of one expert; -inf where it is masked
__device__ __forceinline__ double value64(const RouteArgs& a, const float* row, int e, const Softmax64& sm) {
    const double z = (double)row[e];
    if (z != z || z == neg_inf64()) return neg_inf64();
    const double s = a.o.softmax ? (z == sm.m ? 1.0 : exp(z - sm.m)) / sm.den : 1.0 / (1.0 + exp(-z));
    const double v = a.bias ? s + (double)a.bias[e] : s;
    return v == v ? v : neg_inf64();
}

// Kept groups from 64-bit values: bit g LG for group g.
__device__ __noinline__ unsigned kept_groups64(const RouteArgs& a, const float* row, WarpMem& wm, int LG, int lane) {
    const Softmax64 sm = a.o.softmax ? softmax64(row, a.E, lane) : Softmax64{0.0, 1.0};
    for (int e = lane; e < a.E; e += 32) wm.d[e] = value64(a, row, e, sm);
    __syncwarp();
    const int per = a.E / a.o.groups, my = lane / LG;
    const bool real = my < a.o.groups && my * LG == lane;
    double gv = neg_inf64();
    if (real) {
        double x1 = neg_inf64(), x2 = neg_inf64();
        for (int i = 0; i < per; ++i) {
            const double x = wm.d[my * per + i];
            x2 = fmax(x2, fmin(x1, x));
            x1 = fmax(x1, x);
        }
        gv = a.o.group_top == 2 && x2 != neg_inf64() ? x1 + x2 : x1;
    }
    int ahead = 0;
    for (int g = 0; g < a.o.groups; ++g) {
        const double x = __shfl_sync(kFull, gv, g * LG);
        ahead += x > gv || (x == gv && g < my);
    }
    return __ballot_sync(kFull, real && ahead < a.o.top_groups);
}

// The k best of the n candidates by their 64-bit values, ties to the lower expert.
__device__ __noinline__ void sort_candidates64(const RouteArgs& a, const float* row, WarpMem& wm, int n, int lane) {
    const Softmax64 sm = a.o.softmax ? softmax64(row, a.E, lane) : Softmax64{0.0, 1.0};
    for (int c = lane; c < n; c += 32) wm.d[c] = value64(a, row, wm.cand[c].e, sm);
    __syncwarp();
    for (int c = lane; c < n; c += 32) {
        const double v = wm.d[c];
        const int e = wm.cand[c].e;
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += wm.d[j] > v || (wm.d[j] == v && wm.cand[j].e < e);
        if (rank < a.k) wm.sorted[rank].e = e;
    }
    __syncwarp();
}

// The share of each lane's chosen logit in the sum over the chosen scores
// (lanes without one: live false).  s = e^min(z,0) / (1 + e^-|z|) (sigmoid) or
// e^z / const (softmax), with the largest exponent taken out of the ratio, so
// that it stands where every score underflows.
__device__ __forceinline__ float chosen_share(float z, bool live, bool softmax) {
    const float x = softmax ? z : fminf(z, 0.0f);
    const float m = warp_max(live ? x : neg_inf());
    float p = live ? (x == m ? 1.0f : expf(x - m)) : 0.0f;
    if (!softmax && live) p = __fdividef(p, 1.0f + expf(-fabsf(z)));
    const float tot = warp_sum(p);
    return tot > 0.0f ? __fdividef(p, tot) : 0.0f;
}

__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Issue bound: one token costs a few hundred warp instructions whatever its
// k, and its row only E floats.  So the scores that only decide the choice use
// the hardware's exponential and reciprocal (2 instructions each), and the
// accurate ones are left to the k chosen, one per lane.  A value's low three
// bits are replaced by its register's number j (expert lane + 32 j), so that
// values alone are compared and moved.  Every lane keeps its three best; k + 1
// warp maxima take the best values in descending order, the lane that owns one
// moves its next up.  Where a lane would need its fourth, or two values are
// equal, all values from the threshold found up are compacted and ranked by
// counting instead.
//
// Error bounds, u = 2^-24.  e = 2^(x log2 e): the product's rounding |x| u,
// the hardware's 2 ulp (4u), 1 + e and its reciprocal (3u), for softmax the
// rounding of z - m (|z - m| u) and the product with 1 / sum, whose own error
// is a common factor.  Relative to s: at most (2 |x| + 12) u <= 2^-16.3 (the
// exponential is 0 from |x| = 88 on).  Absolute: (2 * 0.37 + 12) u times the
// largest score (x e^-x <= 0.37), 2^-20.3 each.  Without a bias values are
// compared relatively (the bound counts for both), with one absolutely, plus
// the rounding of v and its low bits, 16u (|v_a| + |v_b|).  A group's value
// sums two.  1e-37 covers what is below the normal range.
constexpr float kRelErr = 0x1p-16f, kAbsErr = 0x1p-19f, kSumErr = 0x1p-20f;

// v with its low three bits replaced by j.
__device__ __forceinline__ float tagged(float v, int j) {
    return __uint_as_float((__float_as_uint(v) & ~7u) | (uint32_t)j);
}

// x1 >= x2 >= x3, the largest so far, with y among them.
__device__ __forceinline__ void insert3(float& x1, float& x2, float& x3, float y) {
    const float t = fminf(x1, y), u = fminf(x2, t);
    x1 = fmaxf(x1, y);
    x2 = fmaxf(x2, t);
    x3 = fmaxf(x3, u);
}

// The best two of each register over the warp: in steps that halve the
// registers, lane l ends with the pair of register l / (32 / VPT).
template <int VPT>
__device__ __forceinline__ void best2_by_register(const float (&v)[VPT], int lane, float& x1, float& x2) {
    float a1[VPT], a2[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        a1[j] = v[j];
        a2[j] = neg_inf();
    }
    int n = VPT;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {  // the upper half of the lanes takes the upper half of the registers
            n /= 2;
            const bool up = lane & o;
#pragma unroll
            for (int j = 0; j < VPT / 2; ++j)
                if (j < n) {
                    const int h = j + n < VPT ? j + n : j;
                    const float y1 = __shfl_xor_sync(kFull, up ? a1[j] : a1[h], o);
                    const float k1 = up ? a1[h] : a1[j];
                    if (o == 16) {  // first step: no second values yet
                        a1[j] = fmaxf(k1, y1);
                        a2[j] = fminf(k1, y1);
                    } else {
                        const float y2 = __shfl_xor_sync(kFull, up ? a2[j] : a2[h], o);
                        const float k2 = up ? a2[h] : a2[j];
                        a2[j] = fmaxf(fminf(k1, y1), fmaxf(k2, y2));
                        a1[j] = fmaxf(k1, y1);
                    }
                }
        } else {
            const float y1 = __shfl_xor_sync(kFull, a1[0], o), y2 = __shfl_xor_sync(kFull, a2[0], o);
            a2[0] = fmaxf(fminf(a1[0], y1), fmaxf(a2[0], y2));
            a1[0] = fmaxf(a1[0], y1);
        }
    }
    x1 = a1[0];
    x2 = a2[0];
}

// The general way to the k + 1 best: all values from cut up, compacted and
// ranked by counting.  Returns whether two of them are equal; n: how many.
template <int VPT>
__device__ __noinline__ bool rank_candidates(const float (&v)[VPT], float cut, int k, WarpMem& wm, int lane, int& n) {
    int mine = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) mine += v[j] >= cut;
    int pos = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, pos, o);
        if (lane >= o) pos += x;
    }
    n = __shfl_sync(kFull, pos, 31);
    pos -= mine;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (v[j] >= cut) wm.cand[pos++] = Cand{v[j], lane + 32 * j};
    if (lane == 0) wm.cand[n].v = neg_inf();
    __syncwarp();
    bool equal = false;
    for (int c = lane; c < n; c += 32) {
        const Cand x = wm.cand[c];
        int rank = 0, upto = 0;
        for (int j = 0; j < n; j += 2) {
            const float4 y = *reinterpret_cast<const float4*>(wm.cand + j);  // two candidates
            rank += (y.x > x.v) + (y.z > x.v);
            upto += (y.x >= x.v) + (y.z >= x.v);
        }
        if (rank <= k) {
            wm.sorted[rank] = x;
            equal |= upto - rank > 1;
        }
    }
    return equal;
}

// Lane l holds experts l, l + 32, ...: the experts of one group lie in as many
// lanes as they can, which keeps the lanes' best values distinct experts of
// the kept groups (with runs of experts in a lane, 4 kept groups of 32 filled
// 16 lanes and left three times the candidates).
template <int VPT, bool SOFTMAX, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 4 : 1) route_logits_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    WarpMem& wm = reinterpret_cast<WarpMem*>(smem)[threadIdx.x >> 5];
    int* hist = reinterpret_cast<int*>(smem + WARPS * sizeof(WarpMem));
    const int tid = threadIdx.x, lane = tid & 31;
    const int E = a.E, k = a.k;
    for (int e = tid; e < E; e += WARPS * 32) hist[e] = 0;
    __syncthreads();

    // Groups.  LG lanes of a warp take a group's values from shared memory;
    // a group of 32 experts is one register of the warp, and its best two
    // values meet by shuffles in LG lanes.
    const bool grouped = a.o.top_groups < a.o.groups;
    const int per = E / a.o.groups;
    const bool in_rows = per == 32 && a.o.groups * 2 > VPT;
    int LG = in_rows ? 32 / VPT : 1;
    if (!in_rows)
        while (2 * LG * a.o.groups <= 32) LG *= 2;
    const int my_group = lane / LG;
    float b[VPT];
    unsigned gbit[VPT];  // the bit of each expert's group (group g: bit g LG)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = lane + 32 * j;
        b[j] = a.bias && e < E ? a.bias[e] : 0.0f;
        if (b[j] != b[j]) {  // masked, and reported
            b[j] = neg_inf();
            report(a.status, kStDeviceCheck);
        }
        b[j] = fminf(b[j], 3.4028235e38f);  // +inf: compared in 64 bits
        gbit[j] = grouped ? 1u << (((e * a.per_inv >> 16) * LG) & 31) : 0u;  // e / per
    }

    for (int t = blockIdx.x * WARPS + (tid >> 5); t < a.T; t += gridDim.x * WARPS) {
        const float* row = a.logits + (size_t)t * E;
        float v[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) v[j] = lane + 32 * j < E ? row[lane + 32 * j] : neg_inf();
        bool bad = false;
        float m = 0.0f, top = 1.0f;  // softmax: the largest logit; a bound of the scores
        if (SOFTMAX) {
            m = neg_inf();
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                bad |= v[j] != v[j];
                v[j] = fmaxf(v[j], neg_inf());  // NaN: masked
                m = fmaxf(m, v[j]);
            }
            m = warp_max(m);
            const float ref = fabsf(m) < __int_as_float(0x7f800000) ? m : 0.0f;
            float part = 0.0f, s[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) s[j] = ex2_fast((v[j] - ref) * 1.4426950408889634f);
            if (m > 3.4e38f)  // logit +inf
#pragma unroll
                for (int j = 0; j < VPT; ++j) s[j] = v[j] == m ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) part += s[j];
            top = rcp_fast(fmaxf(warp_sum(part), 1e-30f));
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const float x = tagged(fmaf(s[j], top, b[j]), j);
                v[j] = v[j] == neg_inf() || b[j] == neg_inf() ? neg_inf() : x;
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                bad |= v[j] != v[j];
                const float x = tagged(rcp_fast(1.0f + ex2_fast(v[j] * -1.4426950408889634f)) + b[j], j);
                v[j] = v[j] > neg_inf() && b[j] > neg_inf() ? x : neg_inf();
            }
        }
        const float abs_err = a.bias ? top * kAbsErr : 0.0f, rel_err = a.bias ? kSumErr : kRelErr;

        if (grouped) {
            float x1 = neg_inf(), x2 = neg_inf();
            if (in_rows) {
                best2_by_register<VPT>(v, lane, x1, x2);
            } else {
                float* all = reinterpret_cast<float*>(wm.d);
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (lane + 32 * j < E) all[lane + 32 * j] = v[j];
                __syncwarp();
                if (my_group < a.o.groups) {
                    const int first = my_group * per, last = first + per;
                    for (int i = first + (lane & (LG - 1)); i < last; i += LG) {
                        const float x = all[i];
                        x2 = fmaxf(x2, fminf(x1, x));
                        x1 = fmaxf(x1, x);
                    }
                }
                for (int o = 1; o < LG; o <<= 1) {
                    const float y1 = __shfl_xor_sync(kFull, x1, o), y2 = __shfl_xor_sync(kFull, x2, o);
                    x2 = fmaxf(fminf(x1, y1), fmaxf(x2, y2));
                    x1 = fmaxf(x1, y1);
                }
            }
            float gv = a.o.group_top == 2 && x2 > neg_inf() ? x1 + x2 : x1;
            // the best groups leave one by one; lo: the last kept, hi: the best left
            bool keep = false;
            float lo = neg_inf();
            for (int r = 0; r < a.o.top_groups; ++r) {
                lo = warp_max(gv);
                if (gv == lo && lo > neg_inf()) {
                    keep = true;
                    gv = neg_inf();
                }
            }
            const float hi = warp_max(gv);
            unsigned kept = __ballot_sync(kFull, keep);  // bit g LG (and the group's other lanes)
            const float gerr = 3.0f * abs_err + 2.0f * rel_err * (fabsf(lo) + fabsf(hi)) + 1e-37f;
            if (__popc(kept) > a.o.top_groups * LG || (hi > neg_inf() && !(lo - hi > gerr)))  // equal, or too close
                kept = kept_groups64(a, row, wm, LG, lane);
#pragma unroll
            for (int j = 0; j < VPT; ++j) v[j] = (kept & gbit[j]) ? v[j] : neg_inf();
        }

        // the k + 1 best in descending order
        float x1 = v[0], x2 = neg_inf(), x3 = neg_inf();
#pragma unroll
        for (int j = 1; j < VPT; ++j) insert3(x1, x2, x3, v[j]);
        __syncwarp();  // the last token's readers are done
        int n = 0, taken = 0;
        float thr = neg_inf();
#pragma unroll 3
        for (int r = 0; r <= k; ++r) {
            const float best = warp_max(x1);
            if (!(best > neg_inf())) {
                thr = neg_inf();
                break;
            }
            thr = best;
            if (x1 == best) {
                wm.sorted[r] = Cand{best, lane};
                x1 = x2;
                x2 = x3;
                x3 = neg_inf();
                ++taken;
            }
            ++n;
        }
        bool close = false;
        if (__reduce_add_sync(kFull, VPT > 3 && taken >= 3 ? 1000 : taken) != n) {
            const float cut = fmaxf(thr - (abs_err + 2.0f * rel_err * fabsf(thr) + 1e-37f), -3.4028235e38f);
            close = rank_candidates<VPT>(v, cut, k, wm, lane, n);
        }
        __syncwarp();
        if (lane < k && lane + 1 < n) {
            const float x = wm.sorted[lane].v, y = wm.sorted[lane + 1].v;
            close |= !(x - y > abs_err + rel_err * (fabsf(x) + fabsf(y)) + 1e-37f);
        }
        const bool live = lane < k && lane < n;
        int e = live ? (int)(__float_as_uint(wm.sorted[lane].v) & 7u) * 32 + (wm.sorted[lane].e & 31) : -1;
        if (__any_sync(kFull, close)) {
            const float cut = fmaxf(thr - (abs_err + 2.0f * rel_err * fabsf(thr) + 1e-37f), -3.4028235e38f);
            rank_candidates<VPT>(v, cut, k, wm, lane, n);
            __syncwarp();
            sort_candidates64(a, row, wm, n, lane);
            if (live) e = wm.sorted[lane].e;
        }
        const float z = live ? row[e] : 0.0f;
        float x;
        if (a.o.renormalize)
            x = chosen_share(z, live, SOFTMAX);
        else
            x = !live ? 0.0f : SOFTMAX ? (z == m ? top : expf(z - m) * top) : __fdividef(1.0f, 1.0f + expf(-z));
        if (lane < k) {
            a.idx[(size_t)t * k + lane] = e;
            a.w[(size_t)t * k + lane] = x * a.o.scale;
            if (live)
                atomicAdd(&hist[e], 1);
            else
                bad = true;
        }
        if (bad) report(a.status, kStDeviceCheck);
    }
    __syncthreads();
    if (gridDim.x == 1) {  // the whole batch in this CTA: no cleared counters needed
        for (int e = tid; e < E; e += WARPS * 32) a.counts[e] = hist[e];
    } else {
        for (int e = tid; e < E; e += WARPS * 32)
            if (hist[e]) atomicAdd(&a.counts[e], hist[e]);
    }
}

// ---------------------------------------------------------------- backward

struct RouteBwdArgs {
    const float* logits;
    const int32_t* idx;
    const float* dw;
    const float* dscores;
    int T, E, k;
    RouteOpts o;
    float* dlogits;
    int* status;
};

constexpr int kBwdWarps = 8;

// DENSE: every expert's score is needed (dscores, or softmax as scored);
// otherwise only the chosen logits are read.
template <int VPT, bool DENSE>
__global__ void __launch_bounds__(kBwdWarps * 32) route_logits_bwd_kernel(const __grid_constant__ RouteBwdArgs a) {
    __shared__ __align__(16) float rows[kBwdWarps][32 * VPT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kBwdWarps + warp;
    if (t >= a.T) return;  // warp-uniform
    const int E = a.E, k = a.k, e0 = lane * VPT;
    const bool vec = (E & 3) == 0, softmax = a.o.softmax;
    const float* row = a.logits + (size_t)t * E;
    float* add = rows[warp];  // what the chosen slots add: to dz, or to ds (softmax as scored)

    float s[VPT], ds[VPT];
    if (DENSE) {
        load_row<VPT>(row, e0, E, vec, neg_inf(), s);
        if (a.dscores)
            load_row<VPT>(a.dscores + (size_t)t * E, e0, E, vec, 0.0f, ds);
        else
#pragma unroll
            for (int j = 0; j < VPT; ++j) ds[j] = 0.0f;
    }
    // chosen slots
    int e = -1;
    float G = 0.0f, z = neg_inf();
    if (lane < k) {
        e = a.idx[(size_t)t * k + lane];
        if (e < -1 || e >= E) {
            report(a.status, kStDeviceCheck);
            e = -1;
        }
        if (e >= 0) {
            G = a.dw[(size_t)t * k + lane] * a.o.scale;
            z = row[e];
        }
    }
    const bool live = e >= 0 && z > neg_inf();  // not masked, not NaN
    float c = 0.0f;
    if (a.o.renormalize) {
        const float p = chosen_share(z, live, softmax);
        const float dot = warp_sum(live ? G * p : 0.0f);
        if (live) c = p * (G - dot) * (softmax ? 1.0f : __fdividef(1.0f, 1.0f + expf(z)));
    } else if (softmax) {
        c = live ? G : 0.0f;
    } else if (live) {
        const float x = expf(-fabsf(z)), y = __fdividef(1.0f, 1.0f + x);
        c = G * x * y * y;
    }
    // an expert listed twice: the first slot takes the sum, in slot order
    const unsigned same = __match_any_sync(kFull, live ? e : -1 - lane);
    bool first = live;
    if (__any_sync(kFull, live && (same & (same - 1)) != 0)) {
        float sum = 0.0f;
        for (int r = 0; r < k; ++r) {
            const float x = __shfl_sync(kFull, c, r);
            if ((same >> r) & 1u) sum += x;
        }
        if (live) c = sum;
        first = live && __ffs(same) - 1 == lane;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) add[lane + 32 * j] = 0.0f;
    __syncwarp();
    if (first) add[e] = c;
    __syncwarp();
    float dz[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) dz[j] = 0.0f;
    load_row<VPT>(add, e0, 32 * VPT, true, 0.0f, dz);
    if (DENSE) {
        if (softmax) {
            float m = neg_inf();
#pragma unroll
            for (int j = 0; j < VPT; ++j) m = fmaxf(m, s[j]);
            m = warp_max(m);
            float part = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const bool in = s[j] > neg_inf();
                s[j] = !in ? 0.0f : s[j] == m ? 1.0f : expf(s[j] - m);
                if (!in) ds[j] = 0.0f;
                if (!a.o.renormalize) {
                    ds[j] += dz[j];
                    dz[j] = 0.0f;
                }
                part += s[j];
                dot += ds[j] * s[j];
            }
            const float inv = __fdividef(1.0f, warp_sum(part));
            dot = warp_sum(dot) * inv;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (s[j] > 0.0f) dz[j] += s[j] * inv * (ds[j] - dot);
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (s[j] > neg_inf()) {
                    const float x = expf(-fabsf(s[j])), y = __fdividef(1.0f, 1.0f + x);
                    dz[j] += ds[j] * x * y * y;
                }
        }
    }
    float* out = a.dlogits + (size_t)t * E;
    if (VPT % 4 == 0 && vec) {
#pragma unroll
        for (int j = 0; j < VPT; j += 4)
            if (e0 + j < E)
                *reinterpret_cast<float4*>(out + e0 + j) =
                    make_float4(dz[j], dz[j + 1 < VPT ? j + 1 : j], dz[j + 2 < VPT ? j + 2 : j], dz[j + 3 < VPT ? j + 3 : j]);
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (e0 + j < E) out[e0 + j] = dz[j];
    }
}

template <int VPT, bool SOFTMAX, int WARPS>
cudaError_t launch_route(const RouteArgs& a, int grid, cudaStream_t st) {
    auto kern = route_logits_kernel<VPT, SOFTMAX, WARPS>;
    constexpr size_t smem = WARPS * sizeof(WarpMem) + kMaxExperts * sizeof(int);
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    kern<<<grid, WARPS * 32, smem, st>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

template <int VPT>
cudaError_t launch_route_v(const RouteArgs& a, int num_sms, cudaStream_t st) {
    if (a.T <= 64)  // one CTA
        return a.o.softmax ? launch_route<VPT, true, 32>(a, 1, st) : launch_route<VPT, false, 32>(a, 1, st);
    const cudaError_t err = cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * (size_t)a.E, st);
    if (err != cudaSuccess) return err;
    const int blocks = (a.T + 7) / 8, grid = blocks < 4 * num_sms ? blocks : 4 * num_sms;
    return a.o.softmax ? launch_route<VPT, true, 8>(a, grid, st) : launch_route<VPT, false, 8>(a, grid, st);
}

template <int VPT>
cudaError_t launch_bwd_v(const RouteBwdArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T + kBwdWarps - 1) / kBwdWarps);
    if (a.dscores || (a.o.softmax && !a.o.renormalize))
        route_logits_bwd_kernel<VPT, true><<<grid, kBwdWarps * 32, 0, st>>>(a);
    else
        route_logits_bwd_kernel<VPT, false><<<grid, kBwdWarps * 32, 0, st>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_logits(const float* logits, const float* bias, int T, int E, int k, const RouteOpts& o,
                                int32_t* idx, float* w, int32_t* counts, int* status, int num_sms, cudaStream_t st) {
    if (T == 0) return cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)E, st);
    const int per = E / o.groups;
    const RouteArgs a{logits, bias, T, E, k, (65536 + per - 1) / per, o, idx, w, counts, status};
    return E <= 32    ? launch_route_v<1>(a, num_sms, st)
           : E <= 64  ? launch_route_v<2>(a, num_sms, st)
           : E <= 128 ? launch_route_v<4>(a, num_sms, st)
                      : launch_route_v<8>(a, num_sms, st);
}

cudaError_t launch_route_logits_bwd(const float* logits, const int32_t* idx, const float* dw, const float* dscores,
                                    int T, int E, int k, const RouteOpts& o, float* dlogits, int* status,
                                    cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const RouteBwdArgs a{logits, idx, dw, dscores, T, E, k, o, dlogits, status};
    return E <= 32    ? launch_bwd_v<1>(a, st)
           : E <= 64  ? launch_bwd_v<2>(a, st)
           : E <= 128 ? launch_bwd_v<4>(a, st)
                      : launch_bwd_v<8>(a, st);
}

}  // namespace moe
