// Routing from gate logits and its gradient ("DeepSeek V3 From Scratch", "In
// code", route(): scores, biased choice, weights from the unbiased scores;
// "Scaling Efficiency: A Deep Dive into the DeepSeek-V3 Architecture",
// DeepSeekMoE sketch: softmax gating), with sigmoid or softmax scores and the
// choice limited to the best groups of experts.
//
// Forward, one warp per token, or per four tokens of a batch:
//   s = sigmoid(z) or softmax(z);  v = s + bias;
//   group value = sum of the group's 1 or 2 largest v; the top_groups best
//   groups are kept (ties: lower group); the k largest v of the kept groups
//   in descending order (ties: lower expert);  w = scale s / (sum of the k s).
// v is defined in 64 bits.  The kernels form it in 32 and bound the error:
// where two values whose order matters are closer than the bound, the values
// concerned are formed again in 64 bits.
//
// Backward, one warp per token or several, for the choice made:  with G = scale dw,
//   renormalised:  dz_j = p_j (G_j - sum G p) (sigmoid: times 1 - s_j), p the
//     chosen scores' shares, whatever the other experts' logits are;
//   as scored:     ds_j += G_j;
//   dense part:    sigmoid  dz = ds s (1 - s),  softmax  dz = s (ds - sum ds s).
#include "common.cuh"
#include "kernels.h"
#include "pdl.h"

#include <cstddef>

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxK = 16;
// Tokens, and CTAs, of a batch that one cluster takes.  A second launch costs the
// host 2 us; on the device the cluster's barriers and reads take 0.3 us longer at
// 128 tokens, 0.6 to 0.9 at 136 to 256.
constexpr int kSmallTokens = 128, kSmallCtas = 8;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ double neg_inf64() { return __longlong_as_double(0xfff0000000000000ll); }

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ int ld_cluster_i32(uint32_t cluster_addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
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
    Cand sorted[kMaxK + 2];       // the k + 1 best, descending (rank_candidates)
    int first[32];                // first expert of each kept group
    int place[kMaxK + 2];         // lane of the r-th best; expert of the r-th by 64-bit values
};
static_assert(sizeof(WarpMem) % 16 == 0, "vector reads in every warp's copy");

struct RouteArgs {
    const float* logits;
    const float* bias;
    int T, E, k;
    int per;           // experts of a group
    int per_inv;       // ceil(2^16 / per): e / per = e per_inv >> 16 for e, per <= 256
    int group_lanes;   // lanes that take a group's values, a power of two
    int direct;        // the kept groups' values are taken where they are, not listed again
    unsigned leaders;  // lane g group_lanes of every group g
    // four tokens per warp: runs of experts (the groups, or all as one) in chunks of four
    int run, run_chunks, chunks;
    int chunk_inv;     // c / run_chunks = c chunk_inv >> 16
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
__device__ __forceinline__ Softmax64 softmax64(const float* row, int E, int lane) {
    constexpr int N = kMaxExperts / 32;
    float z[N], m = neg_inf();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        z[j] = lane + 32 * j < E ? row[lane + 32 * j] : neg_inf();
        m = fmaxf(m, z[j]);  // NaN drops out
    }
    m = warp_max(m);
    double part = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) {  // side by side: one after the other they took 2 us
        const double y = exp((double)z[j] - (double)m);
        part += z[j] == m ? 1.0 : z[j] > neg_inf() ? y : 0.0;
    }
    return {(double)m, warp_sum(part)};
}
// v of one expert; -inf where it is masked
__device__ __forceinline__ double value64(const RouteArgs& a, const float* row, int e, const Softmax64& sm) {
    const double z = (double)row[e];
    if (z != z || z == neg_inf64()) return neg_inf64();
    const double s = a.o.softmax ? (z == sm.m ? 1.0 : exp(z - sm.m)) / sm.den : 1.0 / (1.0 + exp(-z));
    const double v = a.bias ? s + (double)a.bias[e] : s;
    return v == v ? v : neg_inf64();
}

// Kept groups from 64-bit values (bit g LG for group g): of each group, the
// values that may be among its group_top largest are evaluated.  all: the
// 32-bit values; cut: this lane's group's group_top-th, less the error bound.
__device__ __noinline__ unsigned kept_groups64(const RouteArgs& a, const float* row, const float* all, float cut,
                                               int lane) {
    const Softmax64 sm = a.o.softmax ? softmax64(row, a.E, lane) : Softmax64{0.0, 1.0};
    const int LG = a.group_lanes, my = lane / LG;
    const int last = my < a.o.groups ? (my + 1) * a.per : 0;
    double x1 = neg_inf64(), x2 = neg_inf64();
    int i = my * a.per + (lane & (LG - 1));
    for (;;) {  // every lane's next value above its cut, evaluated together
        while (i < last && !(all[i] >= cut)) i += LG;
        if (!__any_sync(kFull, i < last)) break;
        if (i < last) {
            const double x = value64(a, row, i, sm);
            x2 = fmax(x2, fmin(x1, x));
            x1 = fmax(x1, x);
            i += LG;
        }
    }
    for (int o = 1; o < LG; o <<= 1) {
        const double y1 = __shfl_xor_sync(kFull, x1, o), y2 = __shfl_xor_sync(kFull, x2, o);
        x2 = fmax(fmin(x1, y1), fmax(x2, y2));
        x1 = fmax(x1, y1);
    }
    const double gv = a.o.group_top == 2 && x2 != neg_inf64() ? x1 + x2 : x1;
    int ahead = 0;
    for (int g = 0; g < a.o.groups; ++g) {
        const double x = __shfl_sync(kFull, gv, g * LG);
        ahead += x > gv || (x == gv && g < my);
    }
    return __ballot_sync(kFull, gv != neg_inf64() && ahead < a.o.top_groups) & a.leaders;
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
        if (rank < a.k) wm.place[rank] = e;
    }
    __syncwarp();
}

// The lanes' experts (lane r < n: e) in the order of their 64-bit values.
__device__ __noinline__ int reorder64(const RouteArgs& a, const float* row, WarpMem& wm, int e, int n, int lane) {
    const Softmax64 sm = a.o.softmax ? softmax64(row, a.E, lane) : Softmax64{0.0, 1.0};
    const double v = lane < n ? value64(a, row, e, sm) : neg_inf64();
    int rank = 0;
    for (int r = 0; r < n; ++r) {
        const double y = __shfl_sync(kFull, v, r);
        const int f = __shfl_sync(kFull, e, r);
        rank += y > v || (y == v && f < e);
    }
    __syncwarp();
    if (lane < n) wm.place[rank] = e;
    __syncwarp();
    return lane < n ? wm.place[lane] : -1;
}

// The share of each lane's chosen logit in the sum over the chosen scores of
// its SLOTS lanes (lanes without one: live false).  s = e^min(z,0) / (1 +
// e^-|z|) (sigmoid) or e^z / const (softmax), with the largest exponent taken
// out of the ratio, so that it stands where every score underflows.
// __fdividef here and below: 2 ulp instead of half of one, a reciprocal and a
// product.  Its divisors lie between 1 and 256, or are 1 + e^|z|, whose quotient it
// flushes to 0 only below the normal range.
template <int SLOTS>
__device__ __forceinline__ float chosen_share(float z, bool live, bool softmax) {
    const float x = softmax ? z : fminf(z, 0.0f);
    float m = live ? x : neg_inf();
#pragma unroll
    for (int o = SLOTS / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float p = live ? (x == m ? 1.0f : expf(x - m)) : 0.0f;
    if (!softmax && live) p = __fdividef(p, 1.0f + expf(-fabsf(z)));
    float tot = p;
#pragma unroll
    for (int o = SLOTS / 2; o > 0; o >>= 1) tot += __shfl_xor_sync(kFull, tot, o);
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

// Issue bound: one token costs 500 to 700 warp instructions whatever its k,
// and its row only E floats.  So the scores that only decide the choice use
// the hardware's exponential and reciprocal (2 instructions each), and the
// accurate ones are left to the k chosen, one per lane.  A value's low three
// bits are replaced by its register's number j, so that values alone are
// compared and moved.  Every lane sorts its four best; k + 1 warp maxima take the
// best values in descending order, the lane that owns one moves its next up.
// Where a lane would need its fifth, or two values are equal, all values from the
// threshold found up are compacted and ranked by counting instead.
//
// Error bounds, u = 2^-24.  e = 2^(x log2 e): the product's rounding and the
// constant's, 1.3 |x| u, the hardware's 2 ulp (4u), 1 + e and its reciprocal
// (3u), for softmax the rounding of z - m (|z - m| u) and the product with
// 1 / sum.  Relative to s: at most (2.3 |x| + 12) u <= 2^-16.2 (the exponential
// is 0 from |x| = 88 on), the error of 1 / sum left out: without a bias it is a
// factor of every value compared.  Absolute: (2.3 * 0.37 + 4 + 3) u <= 8u times the
// largest score (x e^-x <= 0.37) each, 16u for two; for softmax scores with a bias
// the difference of two also carries the error of 1 / sum: the terms' own, (2.3 |x|
// + 4) u with |x| averaged over the scores (at most 3.4: 255 terms of e^-4.3 beside
// the largest), 7 additions in a lane, 5 across lanes and the reciprocal's 2u, 26u.
// Without a bias values are compared relatively (the bound counts for both), with
// one absolutely, plus the rounding of v and its low bits, 16u (|v_a| + |v_b|).  A
// group's value sums two: see group_span.  1e-37 covers what is below the normal
// range.
constexpr float kRelErr = 0x1p-16f, kAbsErr = 0x1p-19f, kAbsErrSoftmax = 0x1p-18f, kSumErr = 0x1p-20f;
constexpr float kLog2e = 1.4426950408889634f, kFltMax = 3.4028234664e38f;
// A masked value, and the bound below which a value is one.  Finite biases are
// held above it (those beyond kLeastBias tie in 32 bits and are compared in 64).
constexpr float kMasked = -kFltMax, kLow = -1e38f, kLeastBias = -1e37f;

// v with its low bits (three, or those of MASK) replaced by j.
template <uint32_t MASK = 7u>
__device__ __forceinline__ float tagged(float v, int j) {
    return __uint_as_float((__float_as_uint(v) & ~MASK) | (uint32_t)j);
}

__device__ __forceinline__ void order(float& a, float& b) {  // a >= b
    const float t = fminf(a, b);
    a = fmaxf(a, b);
    b = t;
}
__device__ __forceinline__ void sort4(float (&x)[4]) {
    order(x[0], x[1]);
    order(x[2], x[3]);
    order(x[0], x[2]);
    order(x[1], x[3]);
    order(x[1], x[2]);
}
// The four largest so far, descending, and the fifth, with y among them.
__device__ __forceinline__ void insert4(float (&x)[4], float& fifth, float y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) order(x[i], y);
    fifth = fmaxf(fifth, y);
}
// The four largest of v, descending, and the fifth.
template <int VPT>
__device__ __forceinline__ void best4(const float (&v)[VPT], float (&x)[4], float& fifth) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = i < VPT ? v[i < VPT ? i : 0] : kMasked;
    if (VPT == 2) order(x[0], x[1]);
    if (VPT >= 4) sort4(x);
    if (VPT == 8) {
        float y[4] = {v[4 % VPT], v[5 % VPT], v[6 % VPT], v[7 % VPT]};
        sort4(y);
#pragma unroll
        for (int i = 0; i < 4; ++i) order(x[i], y[3 - i]);  // x: the four largest, rising then falling
        fifth = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        order(x[0], x[2]);
        order(x[1], x[3]);
        order(x[0], x[1]);
        order(x[2], x[3]);
    }
}

// The two largest of v, x1 >= x2 (VPT 1: x2 masked).
template <int VPT>
__device__ __forceinline__ void best2(const float (&v)[VPT], float& x1, float& x2) {
    float hi[VPT], lo[VPT];
#pragma unroll
    for (int j = 0; j < VPT / 2; ++j) {
        hi[j] = fmaxf(v[2 * j], v[2 * j + 1 < VPT ? 2 * j + 1 : 0]);
        lo[j] = fminf(v[2 * j], v[2 * j + 1 < VPT ? 2 * j + 1 : 0]);
    }
    if (VPT == 1) {
        hi[0] = v[0];
        lo[0] = kMasked;
    }
#pragma unroll
    for (int n = VPT / 4; n > 0; n /= 2)
#pragma unroll
        for (int j = 0; j < n; ++j) {
            lo[j] = fmaxf(fminf(hi[j], hi[j + n]), fmaxf(lo[j], lo[j + n]));
            hi[j] = fmaxf(hi[j], hi[j + n]);
        }
    x1 = hi[0];
    x2 = lo[0];
}

// Where candidates begin below the (k + 1)-th value found.
__device__ __forceinline__ float cut_of(float best, float abs_err, float rel_err) {
    return fmaxf(best - (abs_err + 2.0f * rel_err * fabsf(best) + 1e-37f), kLow);
}

// What a group may be worth at least and at most, from its best member x1, its
// other one x2 (two) and their 32-bit value gv.  The error is that of the members
// and of the sum's rounding; it follows the members' sizes.  The sum may be far
// smaller, with biases of both signs, so each group is held to its own.  Members
// held above the lowest biases (kLeastBias) may be worth any less, those held at
// the largest number (bias +inf) any more; a sum that is infinite says nothing.
struct Span {
    float least, most;
};
__device__ __forceinline__ Span group_span(float gv, float x1, float x2, bool two, float abs_err, float rel_err) {
    const float off = 1.5f * abs_err + 2.0f * rel_err * (fabsf(x1) + (two ? fabsf(x2) : 0.0f)) + 1e-37f;
    Span s;
    s.least = gv <= kFltMax && (two ? x2 : x1) > 0.9f * kLeastBias ? gv - off : kMasked;
    s.most = x1 < 3.4e38f ? gv + off : kFltMax;
    return s;
}

// The general way to the k + 1 best: all values of the kept groups (bit g LG
// of kept) from cut up, compacted and ranked by counting.  Returns whether two
// of them are equal; n: how many.  More than kManyCandidates (rows of equal
// values) are not ranked: route_token64's k rounds are shorter then (8192 rows of
// 256 equal values: 35 us, by ranking 452).
constexpr int kManyCandidates = 48;
template <bool SOFTMAX>
__device__ __noinline__ void route_token64(const RouteArgs& a, WarpMem& wm, int* hist, int t, int lane);
template <int VPT>
__device__ __noinline__ bool rank_candidates(const RouteArgs& a, const float (&v)[VPT], unsigned kept, int LG, float cut,
                                             WarpMem& wm, int lane, int& n) {
    unsigned in = 0u;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int g = (lane * VPT + j) * a.per_inv >> 16;
        if (v[j] >= cut && ((kept >> ((g * LG) & 31)) & 1u)) in |= 1u << j;
    }
    int pos = __popc(in);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, pos, o);
        if (lane >= o) pos += x;
    }
    n = __shfl_sync(kFull, pos, 31);
    if (n > kManyCandidates) return true;
    pos -= __popc(in);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if ((in >> j) & 1u) wm.cand[pos++] = Cand{v[j], lane * VPT + j};
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
        if (rank <= a.k) {
            wm.sorted[rank] = x;
            equal |= upto - rank > 1;
        }
    }
    return equal;
}

// This lane's biases, as the 32-bit choice takes them; odd: one masks or forces.
template <int VPT>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int lane, float (&b)[VPT], bool& odd) {
    const int E = a.E, e0 = lane * VPT;
    odd = false;
    load_row<VPT>(a.bias ? a.bias : a.logits, e0, a.bias ? E : 0, (E & 3) == 0, 0.0f, b);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (b[j] != b[j]) {  // masked, and reported
            b[j] = neg_inf();
            report(a.status, kStDeviceCheck);
        }
        odd |= fabsf(b[j]) > kFltMax;
        if (b[j] != neg_inf()) b[j] = fmaxf(fminf(b[j], kFltMax), kLeastBias);
        if (e0 + j >= E) b[j] = kMasked;
    }
    odd = __any_sync(kFull, odd);
}

// One token by one warp.  Lane l holds experts [l VPT, (l + 1) VPT).  Grouped choices list the kept
// groups' experts again over all lanes, so that no lane holds many of them.
template <int VPT, bool SOFTMAX>
__device__ __forceinline__ void route_token(const RouteArgs& a, WarpMem& wm, int* hist, const float (&b)[VPT], bool odd,
                                            int t, int lane) {
    const int E = a.E, k = a.k, e0 = lane * VPT;
    const bool vec = (E & 3) == 0;
    // Groups: LG lanes take a group's values, from their registers where a
    // group is a power of two of whole lanes, else from shared memory.
    const bool grouped = a.o.top_groups < a.o.groups;
    const int per = a.per, LG = a.group_lanes;
    const bool in_lanes = LG * VPT == per;
    const int my_group = lane / LG, sub = lane & (LG - 1);
    const bool real = my_group < a.o.groups;
            const float* row = a.logits + (size_t)t * E;
            float v[VPT];
            load_row<VPT>(row, e0, E, vec, kMasked, v);
            float nf = 0.0f;  // NaN where a logit is not finite
    #pragma unroll
            for (int j = 0; j < VPT; ++j) nf = fmaf(v[j], 0.0f, nf);
            bool special = nf != nf;
            float m = 0.0f, top = 1.0f;  // softmax: the largest logit; a bound of the scores
            if (SOFTMAX) {
                m = v[0];
    #pragma unroll
                for (int j = 1; j < VPT; ++j) m = fmaxf(m, v[j]);  // NaN drops out
                m = warp_max(m);
                special |= !(m > kLow);
            }
            special = __any_sync(kFull, special) || odd;  // masks, infinities, NaN: the long way
            bool bad = false;
            unsigned masked = 0u;
            if (special) {
    #pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    bad |= v[j] != v[j];
                    if (!(v[j] > neg_inf()) || b[j] == neg_inf() || e0 + j >= E) masked |= 1u << j;
                    if (!(v[j] > neg_inf()) || e0 + j >= E) v[j] = neg_inf();
                }
            }
            if (SOFTMAX) {
                float part = 0.0f;
                if (special) {
                    const float ref = fabsf(m) <= kFltMax ? m : 0.0f;
    #pragma unroll
                    for (int j = 0; j < VPT; ++j) {
                        const float z = v[j];
                        v[j] = ex2_fast((z - ref) * kLog2e);
                        if (m > kFltMax) v[j] = z == m ? 1.0f : 0.0f;  // logit +inf
                    }
                } else {
    #pragma unroll
                    for (int j = 0; j < VPT; ++j) v[j] = ex2_fast((v[j] - m) * kLog2e);
                }
    #pragma unroll
                for (int j = 0; j < VPT; ++j) part += v[j];
                // also the factor of weights as scored: off by at most 26 units of 2^-24 (see kAbsErrSoftmax), once
                // per weight
                top = rcp_fast(fmaxf(warp_sum(part), 1e-30f));
    #pragma unroll
                for (int j = 0; j < VPT; ++j) v[j] = tagged(fmaf(v[j], top, b[j]), j);
            } else {
    #pragma unroll
                for (int j = 0; j < VPT; ++j) v[j] = tagged(rcp_fast(1.0f + ex2_fast(v[j] * -kLog2e)) + b[j], j);
            }
            if (special)
    #pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if ((masked >> j) & 1u) v[j] = kMasked;
            const float abs_err = a.bias ? top * (SOFTMAX ? kAbsErrSoftmax : kAbsErr) : 0.0f, rel_err = a.bias ? kSumErr : kRelErr;

            float x[4] = {kMasked, kMasked, kMasked, kMasked}, fifth = kMasked;
            unsigned kept = a.leaders;
            if (grouped) {
                float* all = reinterpret_cast<float*>(wm.d);
                const auto put = [&] {  // the row's values where every lane can read them
                    __syncwarp();
                    if (VPT % 4 == 0) {
    #pragma unroll
                        for (int j = 0; j < VPT; j += 4)
                            *reinterpret_cast<float4*>(all + e0 + j) =
                                make_float4(v[j], v[j + 1 < VPT ? j + 1 : j], v[j + 2 < VPT ? j + 2 : j],
                                            v[j + 3 < VPT ? j + 3 : j]);
                    } else {
    #pragma unroll
                        for (int j = 0; j < VPT; ++j) all[e0 + j] = v[j];
                    }
                    __syncwarp();
                };
                float x1 = kMasked, x2 = kMasked;
                if (in_lanes) {
                    best2<VPT>(v, x1, x2);
                } else {
                    put();
                    if (real) {
                        const int last = (my_group + 1) * per;
                        for (int i = my_group * per + sub; i < last; i += LG) {
                            const float y = all[i];
                            x2 = fmaxf(x2, fminf(x1, y));
                            x1 = fmaxf(x1, y);
                        }
                    }
                }
                for (int o = 1; o < LG; o <<= 1) {
                    const float y1 = __shfl_xor_sync(kFull, x1, o), y2 = __shfl_xor_sync(kFull, x2, o);
                    x2 = fmaxf(fminf(x1, y1), fmaxf(x2, y2));
                    x1 = fmaxf(x1, y1);
                }
                const bool two = a.o.group_top == 2 && x2 > kLow;
                float gv = two ? x1 + x2 : x1;
                if (!real) gv = kMasked;
                const Span span = group_span(gv, x1, x2, two, abs_err, rel_err);
                // a group's lanes share the comparison with the others
                int ahead = 0;
                for (int i = 0; i < a.o.groups; i += LG) {
                    const float y = __shfl_sync(kFull, gv, ((i + sub) * LG) & 31);
                    ahead += i + sub < a.o.groups && y > gv;
                }
                for (int o = 1; o < LG; o <<= 1) ahead += __shfl_xor_sync(kFull, ahead, o);
                const bool keep = ahead < a.o.top_groups && gv > kLow;
                kept = __ballot_sync(kFull, keep) & a.leaders;
                // the least that a kept group may be worth against the most that another may
                const float lo = -warp_max(keep ? -span.least : kMasked), hi = warp_max(keep ? kMasked : span.most);
                if (__popc(kept) > a.o.top_groups || (hi > kLow && !(lo > hi))) {
                    if (in_lanes) put();
                    kept = kept_groups64(a, row, all, cut_of(two ? x2 : x1, abs_err, rel_err), lane);
                }
                if (a.direct) {
                    best4<VPT>(v, x, fifth);
                    if (!((kept >> (my_group * LG & 31)) & 1u)) x[0] = x[1] = x[2] = x[3] = fifth = kMasked;
                } else {
                    // the kept groups' experts in a row, 32 at a time
                    if (in_lanes) put();
                    if ((kept >> lane) & 1u) wm.first[__popc(kept & ((1u << lane) - 1u))] = my_group * per;
                    __syncwarp();
                    const int count = __popc(kept) * per;
    #pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (32 * i < count) {
                            const int q = lane + 32 * i, g = q * a.per_inv >> 16;
                            float y = kMasked;
                            if (q < count) y = tagged(all[wm.first[g] + q - g * per], i);
                            insert4(x, fifth, y);
                        }
                }
            } else {
                best4<VPT>(v, x, fifth);
            }

            // the k + 1 best in descending order, the r-th in lane r
            __syncwarp();  // the last token's readers are done
            float best = kMasked, mine = kMasked;
            int taken = 0;
    #pragma unroll
            for (int r = 0; r <= kMaxK; ++r) {
                if (r > k) break;
                best = warp_max(x[0]);
                const bool own = x[0] == best;
                if (own) wm.place[r] = lane;
                if (lane == r) mine = best;
                x[0] = own ? x[1] : x[0];
                x[1] = own ? x[2] : x[1];
                x[2] = own ? x[3] : x[2];
                x[3] = own ? kMasked : x[3];
                taken += own;
            }
            // every round one lane's, and no lane's fifth wanted
            bool close = false, ranked = false;
            int n = k + 1;
            if (__reduce_add_sync(kFull, taken >= 4 && fifth >= best ? 1000 : taken) != k + 1 || !(best > kLow)) {
                close = rank_candidates<VPT>(a, v, kept, LG, cut_of(best, abs_err, rel_err), wm, lane, n);
                ranked = true;
            }
            __syncwarp();
            int e = -1;
            const bool live = lane < k && lane < n;
            if (ranked) {
                if (lane <= k && lane < n) {
                    mine = wm.sorted[lane].v;
                    e = wm.sorted[lane].e;
                }
            } else if (lane < k) {  // the value's lane; its low bits: the register
                const int j = (int)(__float_as_uint(mine) & 7u), from = wm.place[lane];
                if (grouped && !a.direct) {
                    const int q = from + 32 * j, g = q * a.per_inv >> 16;
                    e = wm.first[g] + q - g * per;
                } else {
                    e = from * VPT + j;
                }
            }
            const float next = __shfl_down_sync(kFull, mine, 1);
            const float gap = abs_err + rel_err * (fabsf(mine) + fabsf(next)) + 1e-37f;
            const bool unclear = live && lane + 1 < n && !(mine - next > gap);
            const unsigned pairs = __ballot_sync(kFull, unclear);
            if (pairs || __any_sync(kFull, close)) {
                if (((pairs >> (k - 1)) & 1u) || __any_sync(kFull, close)) {  // who is among the k, too
                    if (!ranked) rank_candidates<VPT>(a, v, kept, LG, cut_of(best, abs_err, rel_err), wm, lane, n);
                    if (n > kManyCandidates) return route_token64<SOFTMAX>(a, wm, hist, t, lane);
                    __syncwarp();
                    sort_candidates64(a, row, wm, n, lane);
                    e = live ? wm.place[lane] : -1;
                } else {
                    e = reorder64(a, row, wm, e, k < n ? k : n, lane);
                }
            }
            if (!live) e = -1;
            const float z = live ? row[e] : 0.0f;
            float wt;
            if (a.o.renormalize)
                wt = k <= 8 ? chosen_share<8>(z, live, SOFTMAX) : chosen_share<16>(z, live, SOFTMAX);
            else
                wt = !live ? 0.0f : SOFTMAX ? (z == m ? top : expf(z - m) * top) : __fdividef(1.0f, 1.0f + expf(-z));
            if (lane < k) {
                a.idx[(size_t)t * k + lane] = e;
                a.w[(size_t)t * k + lane] = wt * a.o.scale;
                if (live)
                    atomicAdd(&hist[e], 1);
                else
                    bad = true;
            }
            if (bad) report(a.status, kStDeviceCheck);
}

// The CTA's counts to all.  SMALL: one cluster takes the batch and adds its
// CTAs' counts itself; otherwise counts were cleared by the kernel before this
// one on the stream.
template <int WARPS, bool SMALL>
__device__ __forceinline__ void finish_counts(const RouteArgs& a, const int* hist, int tid) {
    const int E = a.E;
    if (SMALL) {
        cluster_sync_all();  // every CTA's counts are in
        const unsigned n_ctas = gridDim.x;
        for (int e = blockIdx.x * WARPS * 32 + tid; e < E; e += n_ctas * WARPS * 32) {
            int c = 0;
            for (unsigned r = 0; r < n_ctas; ++r) c += ld_cluster_i32(mapa_shared(smem_u32(hist + e), r));
            a.counts[e] = c;
        }
        cluster_sync_all();  // no CTA leaves while its counts are read
    } else {
        __syncthreads();
        for (int e = tid; e < E; e += WARPS * 32)
            if (hist[e]) atomicAdd(&a.counts[e], hist[e]);
    }
}

template <int VPT, bool SOFTMAX, int WARPS, bool SMALL>
__global__ void __launch_bounds__(WARPS * 32, SMALL ? 1 : 4)
    route_logits_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    WarpMem& wm = reinterpret_cast<WarpMem*>(smem)[threadIdx.x >> 5];
    int* hist = reinterpret_cast<int*>(smem + WARPS * sizeof(WarpMem));
    int* taken_tokens = hist + kMaxExperts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.E;
    for (int e = tid; e < E; e += WARPS * 32) hist[e] = 0;
    if (tid == 0) *taken_tokens = WARPS;
    __syncthreads();
    grid_dependency_wait();  // the logits and biases, and the cleared counters

    float b[VPT];
    bool odd;
    load_bias<VPT>(a, lane, b, odd);

    // The CTA's warps take its tokens (every gridDim.x-th) as they come free: a
    // token that needs 64 bits then holds up one warp alone.
    int t_next;
    for (int t = warp * gridDim.x + blockIdx.x; t < a.T; t = t_next) {
        int i_next = 0;
        if (lane == 0) i_next = atomicAdd(taken_tokens, 1);
        t_next = (int)min((long long)__shfl_sync(kFull, i_next, 0) * gridDim.x + blockIdx.x, (long long)a.T);
        if (t_next < a.T && 32 * lane < E)  // its row, on the way while this one is worked on
            asm volatile("prefetch.global.L1 [%0];" ::"l"(a.logits + (size_t)t_next * E + 32 * lane));
        route_token<VPT, SOFTMAX>(a, wm, hist, b, odd, t, lane);
    }
    finish_counts<WARPS, SMALL>(a, hist, tid);
}

// ---- four tokens per warp ----

// v of a sigmoid gate
__device__ __noinline__ double sigmoid64(float z, float b) { return 1.0 / (1.0 + exp(-(double)z)) + (double)b; }

// One token by one warp with every value in 64 bits: k rounds of the largest.
// 6 us for one token of 256 (11700 cycles, most of them FP64 and 64-bit
// compares in dependence), but 8192 rows of equal values take 35 us in all.
template <bool SOFTMAX>
__device__ __noinline__ void route_token64(const RouteArgs& a, WarpMem& wm, int* hist, int t, int lane) {
    constexpr int N = kMaxExperts / 32;
    const int E = a.E, k = a.k;
    const float* row = a.logits + (size_t)t * E;
    __syncwarp();
    bool bad = false;
    float m = neg_inf();
    double den = 1.0;
    for (int e = lane; e < E; e += 32) {
        const float z = row[e];
        bad |= z != z;
        m = fmaxf(m, z);  // NaN drops out
    }
    if (SOFTMAX) {
        m = warp_max(m);
        double part = 0.0;
#pragma unroll 2
        for (int e = lane; e < E; e += 32) {
            const float z = row[e];
            const double y = z == m ? 1.0 : z > neg_inf() ? exp((double)z - (double)m) : 0.0;
            wm.d[e] = y;
            part += y;
        }
        den = warp_sum(part);
    }
#pragma unroll 2
    for (int e = lane; e < E; e += 32) {
        const float z = row[e], b = a.bias ? a.bias[e] : 0.0f;
        const double v = SOFTMAX ? wm.d[e] / den + (double)b : sigmoid64(z, b);
        wm.d[e] = z > neg_inf() && v == v ? v : neg_inf64();
    }
    __syncwarp();
    unsigned kept = a.leaders;
    const int LG = a.group_lanes;
    if (a.o.top_groups < a.o.groups) {
        const int my = lane / LG, last = my < a.o.groups ? (my + 1) * a.per : 0;
        double x1 = neg_inf64(), x2 = neg_inf64();
        for (int i = my * a.per + (lane & (LG - 1)); i < last; i += LG) {
            const double x = wm.d[i];
            x2 = fmax(x2, fmin(x1, x));
            x1 = fmax(x1, x);
        }
        for (int o = 1; o < LG; o <<= 1) {
            const double y1 = __shfl_xor_sync(kFull, x1, o), y2 = __shfl_xor_sync(kFull, x2, o);
            x2 = fmax(fmin(x1, y1), fmax(x2, y2));
            x1 = fmax(x1, y1);
        }
        const double gv = a.o.group_top == 2 && x2 != neg_inf64() ? x1 + x2 : x1;
        int ahead = 0;
        for (int g = 0; g < a.o.groups; ++g) {
            const double x = __shfl_sync(kFull, gv, g * LG);
            ahead += x > gv || (x == gv && g < my);
        }
        kept = __ballot_sync(kFull, gv != neg_inf64() && ahead < a.o.top_groups) & a.leaders;
    }
    // the values as integers of the same order, 0 where there is none
    unsigned long long key[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        key[j] = 0;
        if (e < E && (kept >> ((e * a.per_inv >> 16) * LG & 31) & 1u)) {
            const long long v = __double_as_longlong(wm.d[e] + 0.0);  // -0 -> 0
            if (v != (long long)0xfff0000000000000ll) key[j] = (unsigned long long)(v ^ (v >> 63 | (1ll << 63)));
        }
    }
    int mine = -1;
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
        unsigned long long x = key[0];
        int e = lane;
#pragma unroll
        for (int j = 1; j < N; ++j)
            if (key[j] > x) {
                x = key[j];
                e = lane + 32 * j;
            }
        const unsigned hi = __reduce_max_sync(kFull, (unsigned)(x >> 32));
        bool own = (unsigned)(x >> 32) == hi;
        const unsigned lo = __reduce_max_sync(kFull, own ? (unsigned)x : 0u);
        if ((hi | lo) == 0u) break;
        own &= (unsigned)x == lo;
        e = (int)__reduce_min_sync(kFull, own ? (unsigned)e : ~0u);  // equal values: the lower expert
        if (lane == r) mine = e;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (e == lane + 32 * j) key[j] = 0;
    }
    const bool live = mine >= 0;
    const float z = live ? row[mine] : 0.0f;
    float wt;
    if (a.o.renormalize)
        wt = k <= 8 ? chosen_share<8>(z, live, SOFTMAX) : chosen_share<16>(z, live, SOFTMAX);
    else
        wt = !live     ? 0.0f
             : SOFTMAX ? (z == m ? 1.0f : expf(z - m)) * (float)(1.0 / den)
                       : __fdividef(1.0f, 1.0f + expf(-z));
    if (lane < k) {
        a.idx[(size_t)t * k + lane] = mine;
        a.w[(size_t)t * k + lane] = wt * a.o.scale;
        if (live)
            atomicAdd(&hist[mine], 1);
        else
            bad = true;
    }
    if (bad) report(a.status, kStDeviceCheck);
    __syncwarp();
}

__device__ __forceinline__ float max8(float v) {  // over the 8 lanes of a token
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T sum8(T v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Warps per CTA and CTAs per SM of a batch: 80 registers for the 32 values of a lane, 64
// for fewer (side by side, inputs in L2: 8192 x 256 sigmoid groups 8.7 us, with 64
// registers 9.3; 32768 x 160 softmax groups 12.1 us, with 80 13.4).  More and smaller CTAs add up
// more counts (one atomic per expert and CTA).  A small batch: one cluster of as
// many CTAs as it fills, one up to 32 tokens (the cluster's barrier and reads
// cost 0.8 us; 4 warps per CTA 0.6 more at 32, 16 warps 0.2 to 1.5 at 64 to 128).
constexpr int kQuadCtas = 2;
__host__ __device__ constexpr int quad_warps(int nch, bool small) { return small ? 8 : nch == 8 ? 12 : 16; }
constexpr int kQuadTops = 81;  // float2 per token: 64 chunks, one gap per run, on shifting banks
static_assert(4 * kQuadTops * sizeof(float2) <= offsetof(WarpMem, sorted), "");

// Eight lanes per token, four tokens per warp: what a warp per token spends on
// reductions, on the rounds of the choice and on the weights serves four.
// Experts come in chunks of four; lane r of a token holds chunks r, r + 8, ..
// (a 128-byte line per token and load).  A chunk never straddles two groups: a
// run whose length is no multiple of four ends with a padded chunk.  Chunks
// are sorted, their two best give the group values (through shared memory), and
// the chunks of the kept groups are merged to the lane's four best.
//
// SCORED: the values compared are sigmoid + bias.  Otherwise (no bias, groups by
// their best expert) they are the logits, whose order is that of the scores.
// Logits z + D and z differ as 64-bit scores where neither underflows (600 below
// 0, or below the largest) and, softmax, D >= 2^-30; sigmoid, e^-z D > 2^-50 (1 +
// e^-z lies on a grid of 2^-52): D >= 2^-30 up to z = 13, 2^-16 up to 20, and
// beyond 13 values that the low bits tell apart differ by 2^-17 at least, at 20
// e^-z D is then 2^-46.
//
// Values too close are compared again by exact logits, or as 64-bit sigmoids, one
// per lane (0.6% of the tokens of 256 normal logits with biases).  What is left
// (closer still, NaN, +inf, too few experts) is done by route_token64, 6 us.
//
// Bound by the chain of one quad's instructions, 1579 of 256 sigmoid experts in
// groups, more than by issue slots (38% busy at 8192 tokens, 57% at 32768 x 160):
// 8192 x 256 sigmoid tokens in groups take 8.7 to 10.5 us, of which about 3 are the
// two launches, 32768 x 256 22, 32768 x 160 softmax tokens in groups, 250
// instructions each, 12.5 to 13.8 (the logits at the copy rate: 1.3, 5.2, 3.3).  A
// warp per token took 1.6 to 3 times as long.
template <int NCH, bool SOFTMAX, bool SCORED, bool SMALL>
__global__ void __launch_bounds__(quad_warps(NCH, SMALL) * 32, SMALL ? 1 : kQuadCtas)
    route_logits_quad_kernel(const __grid_constant__ RouteArgs a) {
    static_assert(!(SOFTMAX && SCORED), "closer values would need the 64-bit sum");
    constexpr int N = 4 * NCH, WARPS = quad_warps(NCH, SMALL);
    constexpr uint32_t kTag = N <= 8 ? 7 : N <= 16 ? 15 : 31;  // low bits that name the register
    // the rounding of v and its low bits, (1 + 2 kTag) 2^-24 < (kTag + 1) 2^-23
    constexpr float kTagErr = (kTag + 1) * 0x1p-23f, kLogitErr = 0x1p-30f;
    constexpr float kSaturated = 20.0f, kUnderflow = -600.0f;
    extern __shared__ __align__(16) uint8_t smem[];
    WarpMem& wm = reinterpret_cast<WarpMem*>(smem)[threadIdx.x >> 5];
    float4* bias = reinterpret_cast<float4*>(smem + WARPS * sizeof(WarpMem));  // by chunk; masked: kMasked
    int* hist = reinterpret_cast<int*>(bias + 8 * NCH);
    const int tid = threadIdx.x, lane = tid & 31, r = lane & 7, first_lane = lane & 24;
    const int E = a.E, k = a.k, chunks = a.chunks;
    for (int e = tid; e < E; e += WARPS * 32) hist[e] = 0;
    grid_dependency_wait();  // the logits and biases, and the cleared counters
    if (SCORED)
        for (int i = tid; i < 8 * N; i += WARPS * 32) {
            const int c = i >> 2, g = c * a.chunk_inv >> 16, off = 4 * (c - g * a.run_chunks) + (i & 3);
            float b = kMasked;
            if (c < chunks && off < a.run) {
                b = a.bias ? a.bias[g * a.run + off] : 0.0f;
                if (b != b) report(a.status, kStDeviceCheck);
                b = b > neg_inf() ? fmaxf(fminf(b, kFltMax), kLeastBias) : kMasked;
            }
            reinterpret_cast<float*>(bias)[i] = b;
        }
    __syncthreads();

    const bool vec = (a.run & 3) == 0, grouped = a.o.top_groups < a.o.groups;
    uint32_t group_of = 0u;  // 4 bits per chunk
#pragma unroll
    for (int i = 0; i < NCH; ++i) group_of |= (uint32_t)((r + 8 * i) * a.chunk_inv >> 16 & 15) << (4 * i);
    // without a bias kRelErr has room for the low bits: (2 x 88 + 12 + 63) 2^-24 < 2^-16
    const float rel_err = !SCORED || a.bias ? kTagErr : kRelErr;
    float2* tops = reinterpret_cast<float2*>(wm.d) + (lane >> 3) * kQuadTops;
    uint8_t* place = reinterpret_cast<uint8_t*>(wm.first) + (lane >> 3) * 16;  // lane of the s-th best
    int* ranked = reinterpret_cast<int*>(wm.sorted) + (lane >> 3) * 9;         // expert of the s-th, compared again
    static_assert(4 * 9 * sizeof(int) <= sizeof(wm.sorted) && 4 * 16 <= sizeof(wm.first), "");
    // the expert of a value found in lane `from`
    const auto expert = [&](float value, int from) {
        const int j = (int)(__float_as_uint(value) & kTag), c = from + 8 * (j >> 2);
        const int g = vec ? 0 : c * a.chunk_inv >> 16;
        return g * a.run + 4 * (c - g * a.run_chunks) + (j & 3);
    };
    // exact logits whose scores' order they do not tell
    const auto too_close = [](double x, double y) {
        return !SCORED && x != y && fabs(x - y) < (!SOFTMAX && fmax(x, y) > 13.0 ? 0x1p-16 : (double)kLogitErr);
    };

    const int quads = (a.T - 1) / 4 + 1;
    for (int q = (tid >> 5) * gridDim.x + blockIdx.x; q < quads; q += gridDim.x * WARPS) {
        const int t = 4 * q + (lane >> 3);
        const bool in = t < a.T;  // else the last token once more, not stored
        const float* row = a.logits + (size_t)(in ? t : a.T - 1) * E;
        float v[N];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = r + 8 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = kMasked;
            if (vec) {
                if (c < chunks) {
                    const float4 x = *reinterpret_cast<const float4*>(row + 4 * c);
                    v[4 * i] = x.x;
                    v[4 * i + 1] = x.y;
                    v[4 * i + 2] = x.z;
                    v[4 * i + 3] = x.w;
                }
            } else {
                const int g = group_of >> (4 * i) & 15, off = 4 * (c - g * a.run_chunks);
                const float* p = row + g * a.run + off;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c < chunks && off + j < a.run) v[4 * i + j] = p[j];
            }
        }
        float nf = 0.0f;  // NaN where a logit is not finite
#pragma unroll
        for (int j = 0; j < N; ++j) nf = fmaf(v[j], 0.0f, nf);
        const bool special = __any_sync(kFull, nf != nf);
        unsigned masked = 0u;
        bool again = false;
        float m = 0.0f, top = 1.0f;  // softmax as scored: the largest logit and its score
        if (special) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                again |= v[j] != v[j] || v[j] > kFltMax;
                if (!(v[j] > neg_inf())) masked |= 1u << j;
            }
        }
        if (SOFTMAX && !a.o.renormalize) {
            m = v[0];
#pragma unroll
            for (int j = 1; j < N; ++j) m = fmaxf(m, v[j]);  // NaN drops out
            m = max8(m);
            again |= !(m > kLow);
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) part += ex2_fast((v[j] - m) * kLog2e);
            top = rcp_fast(fmaxf(sum8(part), 1e-30f));
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            float b[4] = {};
            if (SCORED) *reinterpret_cast<float4*>(b) = bias[r + 8 * i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float& x = v[4 * i + j];
                if (SCORED) x = rcp_fast(1.0f + ex2_fast(x * -kLog2e)) + b[j];
                x = tagged<kTag>(x, 4 * i + j);
            }
        }
        if (special) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (masked >> j & 1u) v[j] = kMasked;
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            order(v[4 * i], v[4 * i + 1]);
            order(v[4 * i + 2], v[4 * i + 3]);
            order(v[4 * i], v[4 * i + 2]);
            order(v[4 * i + 1], v[4 * i + 3]);
            order(v[4 * i + 1], v[4 * i + 2]);
        }
        const float abs_err = !SCORED ? kLogitErr : a.bias ? kAbsErr : 0.0f;

        __syncwarp();  // the last tokens' readers are done
        unsigned kept = 0xffu;
        if (grouped) {
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                if (r + 8 * i < chunks)
                    tops[r + 8 * i + (group_of >> (4 * i) & 15)] = make_float2(v[4 * i], v[4 * i + 1]);
            __syncwarp();
            float x1 = kMasked, x2 = kMasked;
            const bool real = r < a.o.groups;
            const float2* mine = tops + (real ? r : 0) * (a.run_chunks + 1);
            for (int i = 0; i < a.run_chunks; ++i) {
                const float2 y = mine[i];
                if (SCORED) x2 = fmaxf(fminf(x1, y.x), fmaxf(x2, y.y));
                x1 = fmaxf(x1, y.x);
            }
            const bool two = SCORED && a.o.group_top == 2 && x2 > kLow;
            float gv = two ? x1 + x2 : x1;
            if (!real) gv = kMasked;
            const Span span = group_span(gv, x1, x2, two, abs_err, rel_err);
            int ahead = 0;
#pragma unroll
            for (int o = 1; o < 8; ++o) ahead += __shfl_sync(kFull, gv, first_lane | ((r + o) & 7)) > gv;
            bool keep = ahead < a.o.top_groups && gv > kLow;
            kept = __ballot_sync(kFull, keep) >> first_lane & 0xffu;
            // the least that a kept group may be worth against the most that another may
            const float lo = -max8(keep ? -span.least : kMasked), hi = max8(keep ? kMasked : span.most);
            const bool unsure = __popc(kept) > a.o.top_groups || (hi > kLow && !(lo > hi));
            const float least = SOFTMAX && !SCORED ? max8(gv) + kUnderflow : kUnderflow;  // a shuffle: by every lane
            if (!SCORED) again |= hi > kLow && (lo < least || (!SOFTMAX && hi > kSaturated));
            if (__any_sync(kFull, unsure)) {
                // the experts of the group's value, if no third (second) is close to them
                const float cut = cut_of(two ? x2 : x1, abs_err, rel_err);
                const bool any = real && x1 > kLow;
                int found = 0, e1 = 0, e2 = 0;
                for (int i = 0; i < a.run_chunks; ++i) {
                    const float2 y = mine[i];
                    const int e0 = r * a.run + 4 * i;
                    if (any && y.x >= cut) {
                        e2 = e1;
                        e1 = e0 + (int)(__float_as_uint(y.x) & 3u);
                        ++found;
                    }
                    if (any && y.y >= cut) {
                        e2 = e1;
                        e1 = e0 + (int)(__float_as_uint(y.y) & 3u);
                        ++found;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NCH; ++i)
                    if (r + 8 * i < chunks) tops[r + 8 * i + (group_of >> (4 * i) & 15)].x = v[4 * i + 2];
                __syncwarp();
                for (int i = 0; i < a.run_chunks; ++i) found += any && mine[i].x >= cut;
                double x = neg_inf64();
                if (any && SCORED) {
                    x = sigmoid64(row[e1], a.bias ? a.bias[e1] : 0.0f);
                    if (two) x += sigmoid64(row[e2], a.bias ? a.bias[e2] : 0.0f);
                } else if (any) {
                    x = row[e1];
                }
                bool unfit = any && found != (two ? 2 : 1);
                int before = 0;
#pragma unroll 1
                for (int o = 1; o < 8; ++o) {
                    const int g = (r + o) & 7;
                    const double y = __shfl_sync(kFull, x, first_lane | g);
                    before += y > x || (y == x && g < r);
                    unfit |= too_close(x, y);
                }
                again |= unsure && unfit;
                keep = unsure ? any && before < a.o.top_groups : keep;
                kept = __ballot_sync(kFull, keep) >> first_lane & 0xffu;
            }
        }
        float x[4];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const float out = kept >> (group_of >> (4 * i) & 15) & 1u ? 0.0f : neg_inf();
            if (i == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = v[j] + out;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = fmaxf(x[j], v[4 * i + 3 - j] + out);
                order(x[0], x[2]);
                order(x[1], x[3]);
                order(x[0], x[1]);
                order(x[2], x[3]);
            }
        }

        // the k + 1 best in descending order, the s-th in lane s
        float best = kMasked, mine = kMasked;
        int taken = 0;
#pragma unroll 1
        for (int s = 0; s <= k; ++s) {
            best = max8(x[0]);
            const bool own = x[0] == best && best > kLow;
            if (own) place[s] = (uint8_t)r;
            if (r == s) mine = best;
            x[0] = own ? x[1] : x[0];
            x[1] = own ? x[2] : x[1];
            x[2] = own ? x[3] : x[2];
            x[3] = own ? kMasked : x[3];
            taken += own;
            if (__any_sync(kFull, own && taken >= 4 && s < k)) {  // a lane without any left takes its next best
                float y = kMasked;
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const float out = kept >> (group_of >> (4 * i) & 15) & 1u ? 0.0f : neg_inf();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float u = v[4 * i + j] + out;
                        if (u < best) y = fmaxf(y, u);
                    }
                }
                if (own && taken >= 4) x[0] = y;
            }
        }
        best = fmaxf(best, kMasked);
        // every round one lane's (the last may find no expert left).  Equal values of two lanes leave a later round
        // empty, and the sum may come out right all the same where no more than k experts stand.
        again |= sum8(taken) != k + (best > kLow) || (r < k && !(mine > kLow));
        float next = __shfl_down_sync(kFull, mine, 1);
        if (r == k - 1) next = best;
        if (!SCORED) {
            const float least = SOFTMAX ? __shfl_sync(kFull, mine, first_lane) + kUnderflow : kUnderflow;
            again |= r < k && (mine < least || (!SOFTMAX && mine > kSaturated));
        }
        const bool close = r < k && !(mine - next > abs_err + rel_err * (fabsf(mine) + fabsf(next)) + 1e-37f);
        unsigned redo = __ballot_sync(kFull, again && in);
        __syncwarp();
        bool live = r < k && in && (redo >> first_lane & 0xffu) == 0u;
        int e = live ? expert(mine, place[r]) : 0;
        if (__any_sync(kFull, close && live)) {
            // the k, and the next where it is close to the last, by what their order is defined on
            const bool sure = !__any_sync(kFull, close && live && r == k - 1);
            bool border = false, unfit = false;
            int en = 0;
            if (!sure) {
                border = (__ballot_sync(kFull, close && live && r == k - 1) >> first_lane & 0xffu) != 0u;
                const float cut = cut_of(best, abs_err, rel_err);
                int all = 0;  // values that may be among the k
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const float out = kept >> (group_of >> (4 * i) & 15) & 1u ? 0.0f : neg_inf();
#pragma unroll
                    for (int j = 0; j < 4; ++j) all += v[4 * i + j] + out >= cut;
                }
                unfit = sum8(all) != k + 1 && border;
                border &= !unfit;
                if (border) en = expert(best, place[k]);
            }
            double u = row[e], n = row[en];
            if (SCORED) {
                u = sigmoid64((float)u, a.bias ? a.bias[e] : 0.0f);
                if (!sure) n = sigmoid64((float)n, a.bias ? a.bias[en] : 0.0f);
            }
            int rank = 0;
#pragma unroll 1
            for (int s = 0; s < k; ++s) {
                const double y = __shfl_sync(kFull, u, first_lane | s);
                const int f = __shfl_sync(kFull, e, first_lane | s);
                rank += y > u || (y == u && f < e);
                unfit |= r < k && too_close(u, y);
            }
            const bool behind = border && r < k && (n > u || (n == u && en < e));  // the next one overtakes it
            unfit |= border && r < k && too_close(u, n);
            rank += behind;
            const int overtaken = __popc(__ballot_sync(kFull, behind) >> first_lane & 0xffu);
            if (r < k && rank < k) ranked[rank] = e;
            if (r == 0 && overtaken > 0) ranked[k - overtaken] = en;
            __syncwarp();
            if (live) e = ranked[r];
            redo |= __ballot_sync(kFull, unfit && in);
            live &= (redo >> first_lane & 0xffu) == 0u;
            if (!live) e = 0;
            __syncwarp();
        }
        const float z = live ? row[e] : 0.0f;
        float wt;
        if (a.o.renormalize)
            wt = chosen_share<8>(z, live, SOFTMAX);
        else
            wt = !live ? 0.0f : SOFTMAX ? (z == m ? top : expf(z - m) * top) : __fdividef(1.0f, 1.0f + expf(-z));
        if (live) {
            a.idx[(size_t)t * k + r] = e;
            a.w[(size_t)t * k + r] = wt * a.o.scale;
            atomicAdd(&hist[e], 1);
        }
        for (unsigned rest = redo; rest;) {  // warp-uniform
            const int which = (__ffs(rest) - 1) >> 3;
            rest &= ~(0xffu << (8 * which));
            route_token64<SOFTMAX>(a, wm, hist, 4 * q + which, lane);
        }
    }
    finish_counts<WARPS, SMALL>(a, hist, tid);
}

// Clears the counters.  The routing kernel's CTAs take their places meanwhile;
// they wait for this kernel's end, and with it for all before it, before they
// read or add anything (reading beside it instead took the same time).
__global__ void clear_counts_kernel(int32_t* counts, int E) {
    grid_dependency_wait();
    grid_launch_dependents();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[e] = 0;
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

// Every expert's score is needed (dscores, or softmax as scored).
template <int VPT>
__global__ void __launch_bounds__(kBwdWarps * 32) route_logits_bwd_kernel(const __grid_constant__ RouteBwdArgs a) {
    __shared__ __align__(16) float rows[kBwdWarps][32 * VPT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kBwdWarps + warp;
    if (t >= a.T) return;  // warp-uniform
    const int E = a.E, k = a.k, e0 = lane * VPT;
    const bool vec = (E & 3) == 0, softmax = a.o.softmax;
    grid_dependency_wait();
    const float* row = a.logits + (size_t)t * E;
    float* add = rows[warp];  // what the chosen slots add: to dz, or to ds (softmax as scored)

    float s[VPT], ds[VPT];
    load_row<VPT>(row, e0, E, vec, neg_inf(), s);
    if (a.dscores)
        load_row<VPT>(a.dscores + (size_t)t * E, e0, E, vec, 0.0f, ds);
    else
#pragma unroll
        for (int j = 0; j < VPT; ++j) ds[j] = 0.0f;
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
        const float p = chosen_share<32>(z, live, softmax);
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

// Only the chosen logits matter (no dscores, and sigmoid or renormalised).
// SLOTS lanes per token, 32 / SLOTS tokens per warp: their rows lie one after
// the other, the warp clears them as one run while the chosen logits arrive,
// then stores the chosen gradients over the zeros.  HBM bound: the rows
// written (putting them together in shared memory first, so that the writes
// started after the gathered reads, took 14.4 instead of 12.2 us at 32768 x 256).
template <int SLOTS>
__global__ void __launch_bounds__(kBwdWarps * 32) route_logits_bwd_chosen_kernel(const __grid_constant__ RouteBwdArgs a) {
    constexpr int TOK = 32 / SLOTS;
    const int lane = threadIdx.x & 31, slot = lane & (SLOTS - 1);
    const int t0 = (blockIdx.x * kBwdWarps + (threadIdx.x >> 5)) * TOK;
    if (t0 >= a.T) return;  // warp-uniform
    const int E = a.E, k = a.k, t = t0 + lane / SLOTS;
    const bool softmax = a.o.softmax;
    int e = -1;
    float G = 0.0f, z = neg_inf();
    grid_dependency_wait();
    if (slot < k && t < a.T) {
        e = a.idx[(size_t)t * k + slot];
        G = a.dw[(size_t)t * k + slot];
    }
    float* out = a.dlogits + (size_t)t0 * E;
    const int count = min(TOK, a.T - t0) * E;
    if ((TOK * E & 3) == 0) {  // every warp's run starts 16-byte aligned
        for (int i = 4 * lane; i + 3 < count; i += 128)
            *reinterpret_cast<float4*>(out + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = (count & ~3) + lane; i < count; i += 32) out[i] = 0.0f;
    } else {
        for (int i = lane; i < count; i += 32) out[i] = 0.0f;
    }
    if (e < -1 || e >= E) {
        report(a.status, kStDeviceCheck);
        e = -1;
    }
    if (e >= 0) z = a.logits[(size_t)t * E + e];
    G = e >= 0 ? G * a.o.scale : 0.0f;
    const bool live = e >= 0 && z > neg_inf();  // not masked, not NaN
    float c = 0.0f;
    if (a.o.renormalize) {
        const float p = chosen_share<SLOTS>(z, live, softmax);
        float dot = live ? G * p : 0.0f;
#pragma unroll
        for (int o = SLOTS / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        if (live) c = p * (G - dot) * (softmax ? 1.0f : __fdividef(1.0f, 1.0f + expf(z)));
    } else if (live) {
        const float x = expf(-fabsf(z)), y = __fdividef(1.0f, 1.0f + x);
        c = G * x * y * y;
    }
    // an expert listed twice: the first slot takes the sum, in slot order
    const int at = lane / SLOTS * E + e;
    const unsigned same = __match_any_sync(kFull, live ? at : -1 - lane);
    bool first = live;
    if (__any_sync(kFull, live && (same & (same - 1)) != 0)) {
        float sum = 0.0f;
        for (int r = 0; r < 32; ++r) {
            const float x = __shfl_sync(kFull, c, r);
            if ((same >> r) & 1u) sum += x;
        }
        if (live) c = sum;
        first = live && __ffs(same) - 1 == lane;
    }
    __syncwarp();  // the warp's zeros are ordered before its gradients
    if (first) out[at] = c;
}

template <int VPT, bool SOFTMAX, int WARPS, bool SMALL>
cudaError_t launch_route(const RouteArgs& a, int grid, cudaStream_t st) {
    constexpr auto kern = route_logits_kernel<VPT, SOFTMAX, WARPS, SMALL>;
    constexpr size_t smem = WARPS * sizeof(WarpMem) + (kMaxExperts + 4) * sizeof(int);
    cudaError_t err = allow_smem<kern>(smem);
    if (err != cudaSuccess) return err;
    note_launches(1);
    return launch_after(kern, dim3((unsigned)grid), WARPS * 32, smem, SMALL ? grid : 1, st, a);
}

template <int VPT>
cudaError_t launch_route_v(const RouteArgs& a, int num_sms, cudaStream_t st) {
    // A token per warp of one cluster, of one CTA up to 8 tokens (3.8 us; a cluster
    // of 8 4.8).  From 9 tokens on the launch that clears the counts and the other
    // form take as long or less on the device (64 tokens 5.6 us against 6.0), but
    // the host needs 2 us more for a second launch.
    constexpr int kSmallWarps = kSmallTokens / kSmallCtas;
    if (a.T <= kSmallTokens) {
        const int grid = a.T <= 8 ? 1 : kSmallCtas;
        if (a.T <= 8 * kSmallCtas)
            return a.o.softmax ? launch_route<VPT, true, 8, true>(a, grid, st)
                               : launch_route<VPT, false, 8, true>(a, grid, st);
        return a.o.softmax ? launch_route<VPT, true, kSmallWarps, true>(a, grid, st)
                           : launch_route<VPT, false, kSmallWarps, true>(a, grid, st);
    }
    note_launches(1);
    const cudaError_t err = launch_after(clear_counts_kernel, dim3(1), 256, 0, 1, st, a.counts, a.E);
    if (err != cudaSuccess) return err;
    const int blocks = (a.T - 1) / 8 + 1, grid = blocks < 4 * num_sms ? blocks : 4 * num_sms;
    return a.o.softmax ? launch_route<VPT, true, 8, false>(a, grid, st) : launch_route<VPT, false, 8, false>(a, grid, st);
}

template <int NCH, bool SOFTMAX, bool SCORED, bool SMALL>
cudaError_t launch_quad_s(const RouteArgs& a, int num_sms, cudaStream_t st) {
    constexpr auto kern = route_logits_quad_kernel<NCH, SOFTMAX, SCORED, SMALL>;
    constexpr int WARPS = quad_warps(NCH, SMALL);
    constexpr size_t smem = WARPS * sizeof(WarpMem) + 8 * NCH * sizeof(float4) + kMaxExperts * sizeof(int);
    cudaError_t err = allow_smem<kern>(smem);
    if (err != cudaSuccess) return err;
    const int quads = (a.T - 1) / 4 + 1;
    if (SMALL) {
        const int grid = (quads - 1) / WARPS + 1;
        note_launches(1);
        return launch_after(kern, dim3((unsigned)grid), WARPS * 32, smem, grid, st, a);
    }
    note_launches(2);
    err = launch_after(clear_counts_kernel, dim3(1), 256, 0, 1, st, a.counts, a.E);
    if (err != cudaSuccess) return err;
    // over all SMs first, then more warps of each: rounds of one quad per warp of an SM's CTA
    const int rounds = (quads - 1) / (WARPS * num_sms) + 1;
    const int grid = quads < num_sms ? quads : (rounds < kQuadCtas ? rounds : kQuadCtas) * num_sms;
    return launch_after(kern, dim3((unsigned)grid), WARPS * 32, smem, 1, st, a);
}

template <int NCH>
cudaError_t launch_quad(const RouteArgs& a, bool scored, int num_sms, cudaStream_t st) {
    const bool small = a.T <= kSmallTokens;
    if (scored)
        return small ? launch_quad_s<NCH, false, true, true>(a, num_sms, st)
                     : launch_quad_s<NCH, false, true, false>(a, num_sms, st);
    if (a.o.softmax)
        return small ? launch_quad_s<NCH, true, false, true>(a, num_sms, st)
                     : launch_quad_s<NCH, true, false, false>(a, num_sms, st);
    return small ? launch_quad_s<NCH, false, false, true>(a, num_sms, st)
                 : launch_quad_s<NCH, false, false, false>(a, num_sms, st);
}

template <int VPT>
cudaError_t launch_bwd_v(const RouteBwdArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T - 1) / kBwdWarps + 1);
    note_launches(1);
    return launch_after(route_logits_bwd_kernel<VPT>, dim3(grid), kBwdWarps * 32, 0, 1, st, a);
}

template <int SLOTS>
cudaError_t launch_bwd_chosen(const RouteBwdArgs& a, cudaStream_t st) {
    constexpr int per_cta = kBwdWarps * 32 / SLOTS;
    note_launches(1);
    return launch_after(route_logits_bwd_chosen_kernel<SLOTS>, dim3((unsigned)((a.T - 1) / per_cta + 1)),
                        kBwdWarps * 32, 0, 1, st, a);
}

}  // namespace

cudaError_t launch_route_logits(const float* logits, const float* bias, int T, int E, int k, const RouteOpts& o,
                                int32_t* idx, float* w, int32_t* counts, int* status, int num_sms, cudaStream_t st) {
    if (T == 0) return cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)E, st);
    const bool grouped = o.top_groups < o.groups;
    const int run = grouped ? E / o.groups : E, run_chunks = (run + 3) / 4, chunks = run_chunks * (E / run);
    // Four tokens per warp (us for 8, 32, 64, 128, 512, 1024, 2048, 3500 tokens, a
    // warp per token against four: 256 experts sigmoid with bias in groups 3.8 5.5 5.7
    // 6.2 5.8 7.3 7.5 8.7, 4.2 5.7 6.3 6.5 6.1 6.4 6.5 6.8; 256 experts softmax 3.4 4.2 4.3
    // 5.0 4.5 6.8 7.7 8.7, 3.5 3.8 4.7 4.7 4.6 4.9 5.1 5.5; 64 experts sigmoid with bias 2.6
    // 3.4 4.3 4.5 4.8 4.8 5.0 6.2, 2.8 3.0 4.3 4.3 4.4 4.5 4.5 4.7; 64 experts softmax 2.7
    // 3.4 3.5 6.9 6.1 6.1 6.1 7.4, 2.6 2.8 3.5 3.6 3.9 4.0 4.0 4.0).  Softmax with a bias or
    // sums of two stays with a warp per token: its close values need the sum in
    // 64 bits, and a quad waits 6 us for that (4096 x 256: 13.0 us against 10.3).
    const bool scored = bias || (grouped && o.group_top == 2);
    const bool quad = T > (scored && chunks > 32 ? kSmallTokens : 8) && !(scored && o.softmax) && k <= 8 &&
                      (!grouped || o.groups <= 8) && chunks <= 64;
    const int vpt = E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : 8;  // experts per lane
    const int per = E / o.groups, whole = per % vpt == 0 ? per / vpt : 0;
    int lanes = whole > 0 && (whole & (whole - 1)) == 0 ? whole : 1;
    if (whole != lanes)
        while (2 * lanes * o.groups <= 32) lanes *= 2;
    unsigned leaders = 0u;
    for (int g = 0; g < o.groups; ++g) leaders |= 1u << (g * lanes);
    // Kept groups that fill at least 16 lanes are taken where they are: the
    // best k + 1 then ask a lane of 8 experts for a fifth in 0.2% of the tokens.
    const bool direct = lanes * vpt == per && (vpt <= 4 || o.top_groups * lanes >= 16);
    const RouteArgs a{logits, bias,   T,      E, k, per, (65536 + per - 1) / per, lanes,
                      direct, leaders, run, run_chunks, chunks, (65536 + run_chunks - 1) / run_chunks, o, idx, w, counts,
                      status};
    if (quad) switch ((chunks + 7) / 8) {  // chunks per lane
            case 1:
            case 2: return launch_quad<2>(a, scored, num_sms, st);
            case 3: return launch_quad<3>(a, scored, num_sms, st);
            case 4: return launch_quad<4>(a, scored, num_sms, st);
            case 5: return launch_quad<5>(a, scored, num_sms, st);
            case 6: return launch_quad<6>(a, scored, num_sms, st);
            default: return launch_quad<8>(a, scored, num_sms, st);
        }
    switch (vpt) {
        case 1: return launch_route_v<1>(a, num_sms, st);
        case 2: return launch_route_v<2>(a, num_sms, st);
        case 4: return launch_route_v<4>(a, num_sms, st);
        default: return launch_route_v<8>(a, num_sms, st);
    }
}

cudaError_t launch_route_logits_bwd(const float* logits, const int32_t* idx, const float* dw, const float* dscores,
                                    int T, int E, int k, const RouteOpts& o, float* dlogits, int* status,
                                    cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const RouteBwdArgs a{logits, idx, dw, dscores, T, E, k, o, dlogits, status};
    if (!dscores && (!o.softmax || o.renormalize))
        return k <= 8 ? launch_bwd_chosen<8>(a, st) : launch_bwd_chosen<16>(a, st);
    return E <= 32    ? launch_bwd_v<1>(a, st)
           : E <= 64  ? launch_bwd_v<2>(a, st)
           : E <= 128 ? launch_bwd_v<4>(a, st)
                      : launch_bwd_v<8>(a, st);
}

}  // namespace moe
