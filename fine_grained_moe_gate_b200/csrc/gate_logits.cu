// Gate logits z = x W_gate^T of a bf16 layer, fp32 ("DeepSeek V3 From
// Scratch", "In code", route(): x @ gate_w.T), on the tensor cores.
//
// A tile = 128 tokens in one CTA, or 256 tokens in a CTA pair (cta_group::2,
// each CTA loads its tokens and half of the W_gate rows), by a chunk of the
// experts; the accumulator is 128 TMEM lanes (tokens) x the chunk's columns.
// K streams through a TMA ring as deep as shared memory holds.  Batches that
// fill too few SMs split K over the CTAs (or pairs) of a cluster, whose
// partial sums meet in the fixed order 0..C-1 through distributed shared
// memory, and the experts over chunks: a decoding step of 64 tokens (d = 7168,
// 256 experts) is bound by what one SM can take in and by latency: 6.4 us (8
// slices of one chunk took 11.3, of 8 chunks 6.8 in the same run).  Large batches
// are HBM bound: x is read once (8192 x 7168: 117 MB, 18.2 us at the copy rate; the
// kernel takes 28.4, the difference is its start, the exchange of the two K halves
// and the store; its 32 tiles of two K halves fill 128 of 148 SMs).
#include "common.cuh"
#include "kernels.h"
#include "pdl.h"
#include "tmap.h"

#include <atomic>

namespace moe {
namespace {

constexpr int BM = 128, BK = 64;
constexpr int A_BYTES = BM * BK * 2;  // 16 KB
constexpr int MAX_STAGES = 12;
// Warps 0 and 2 load x and W_gate, 1 issues the MMAs and owns TMEM; all take
// part in the finish, which moves twice as much in a pair.
template <bool PAIR>
__host__ __device__ constexpr int n_threads() {
    return PAIR ? 512 : 256;
}

struct Ctl {
    uint64_t full[MAX_STAGES];
    uint64_t empty[MAX_STAGES];
    uint64_t tfull;
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
constexpr size_t SMEM_LIMIT = 232448;
constexpr size_t RING_LIMIT = (SMEM_LIMIT - 1024 - sizeof(Ctl)) / 1024 * 1024;

struct GateParams {
    float* z;
    int T, E;
    int n_sub;          // experts of a chunk (a multiple of 16)
    int x_rows;         // token rows of a box: 128, or fewer where the batch is one smaller tile
    uint32_t tmem_cols;
    int k_blocks;
    int stages;
    int ctl_offset;     // of Ctl behind the ring / the partial sums
    int* status;
};

// Row stride (floats) of the partial sums: 16-byte aligned rows on shifting banks.
__host__ __device__ constexpr int part_stride(int n_sub) { return n_sub + 4; }

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// Four logits of a token at expert e (multiples of 4), as many as the row has.
__device__ __forceinline__ void store4(float* row, int e, int E, float4 v) {
    if ((E & 3) == 0) {
        if (e < E) *reinterpret_cast<float4*>(row + e) = v;
    } else {
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < E) row[e + i] = f[i];
    }
}

// Cluster of C CTAs, or of 2C CTAs whose ranks 2c and 2c + 1 are the pair of K
// slice c (the even one issues the MMAs; the odd one holds tokens 128..255 of
// the tile and the upper half of the chunk's W_gate rows).
template <int C, bool PAIR>
__global__ void __launch_bounds__(n_threads<PAIR>(), 1)
    gate_logits_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const GateParams p) {
    constexpr int CL = PAIR ? 2 * C : C, NTHREADS = n_threads<PAIR>();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctl* ctl = reinterpret_cast<Ctl*>(base + p.ctl_offset);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = CL > 1 ? (int)cluster_ctarank() : 0;
    const int half = PAIR ? (crank & 1) : 0;
    const int slice = PAIR ? (crank >> 1) : crank;
    const uint32_t leader = (uint32_t)(crank - half);
    const uint16_t pair_mask = (uint16_t)(3u << leader);
    const int t0 = (int)(blockIdx.x / CL) * (PAIR ? 2 * BM : BM) + half * BM;
    const int e_base = (int)blockIdx.y * p.n_sub;
    const int n_rows = PAIR ? p.n_sub / 2 : p.n_sub;  // W_gate rows this CTA loads per stage
    const int stage_bytes = A_BYTES + n_rows * BK * 2;
    const int kb0 = slice * p.k_blocks / C, kb1 = (slice + 1) * p.k_blocks / C;

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        mbar_init(&ctl->tfull, 1);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(&ctl->tmem_base, p.tmem_cols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&ctl->tmem_base, p.tmem_cols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync_all();  // the leader's barriers are initialised before the peer's loads count on them
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    grid_dependency_wait();
    // both CTAs' parts for a pair; rows of the A tile that no box fills only reach TMEM lanes that are not stored
    const uint32_t stage_tx = (uint32_t)(PAIR ? 2 : 1) * (uint32_t)((p.x_rows + n_rows) * BK * 2);

    if (warp == 0 || warp == 2) {
        const bool tok = warp == 0;  // token boxes (and the arming of the stage), or W_gate boxes
        if (elect_one()) {
            tma_prefetch_desc(tok ? &tmX : &tmW);
            const uint32_t leader_full = PAIR ? mapa_shared(smem_u32(&ctl->full[0]), leader) : 0u;
            int stage = 0;
            uint32_t phase = 0, issued = 0, iss_phase = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, &ctl->abort, p.status)) {
                    ok = false;
                    break;
                }
                uint8_t* a = base + stage * stage_bytes;
                if (PAIR) {
                    if (tok && half == 0) mbar_arrive_expect_tx(&ctl->full[stage], stage_tx);
                    const uint32_t fb = leader_full + 8u * (uint32_t)stage;
                    if (tok)
                        tma_load_2d_pair(a, &tmX, fb, kb * BK, t0, kEvictFirst);
                    else
                        tma_load_2d_pair(a + A_BYTES, &tmW, fb, kb * BK, e_base + half * n_rows, kEvictLast);
                } else {
                    uint64_t* fb = &ctl->full[stage];
                    if (tok) {
                        mbar_arrive_expect_tx(fb, stage_tx);
                        tma_load_2d(a, &tmX, fb, kb * BK, t0, kEvictFirst);
                    } else {
                        tma_load_2d(a + A_BYTES, &tmW, fb, kb * BK, e_base, kEvictLast);
                    }
                }
                issued |= 1u << stage;
                iss_phase = (iss_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                if (PAIR) {
                    settle_inflight_loads();
                } else {
                    for (int s = 0; s < p.stages; ++s)
                        if ((issued >> s) & 1u) mbar_wait_drain(&ctl->full[s], (iss_phase >> s) & 1u);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if ((!PAIR || half == 0) && elect_one()) {
            const uint32_t idesc = idesc_bf16_f32(PAIR ? 2 * BM : BM, p.n_sub);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&ctl->full[stage], phase, &ctl->abort, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint8_t* a = base + stage * stage_bytes;
                const uint64_t ad = smem_desc_sw128(smem_u32(a)), bd = smem_desc_sw128(smem_u32(a + A_BYTES));
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {
                    const uint32_t acc = (kb > kb0 || kk > 0) ? 1u : 0u;
                    if (PAIR)
                        tc_mma_bf16_pair(tmem_base, ad + (uint64_t)(2 * kk), bd + (uint64_t)(2 * kk), idesc, acc);
                    else
                        tc_mma_bf16(tmem_base, ad + (uint64_t)(2 * kk), bd + (uint64_t)(2 * kk), idesc, acc);
                }
                if (PAIR)
                    tc_commit_pair(&ctl->empty[stage], pair_mask);
                else
                    tc_commit(&ctl->empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok) {
                if (PAIR)
                    tc_commit_pair(&ctl->tfull, pair_mask);
                else
                    tc_commit(&ctl->tfull);
            } else {
                if (PAIR)
                    tc_commit_pair(&ctl->drain, (uint16_t)(1u << leader));
                else
                    tc_commit(&ctl->drain);
                mbar_wait_drain(&ctl->drain, 0);
            }
        }
        __syncwarp();
    }

    // TMEM lane r = token r; warp w reads lane quarter w % 4, 16 columns of NTHREADS / 8 at w / 4
    const int q = warp & 3, r = q * 32 + lane;
    float* part = reinterpret_cast<float*>(base);  // C > 1: [128 tokens][part_stride], over the ring
    const int ps = part_stride(p.n_sub);
    const int n_here = p.E - e_base;  // experts the chunk has (may be more than n_sub)
    if (mbar_wait(&ctl->tfull, 0, &ctl->abort, p.status)) {
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
        for (int c = 16 * (warp >> 2); c < p.n_sub; c += NTHREADS / 8) {
            uint32_t v[16];
            tmem_ld16(taddr + (uint32_t)c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                             __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
                if (C > 1)
                    *reinterpret_cast<float4*>(part + r * ps + c + 4 * i) = f;
                else if (t0 + r < p.T)
                    store4(p.z + (size_t)(t0 + r) * p.E, e_base + c + 4 * i, p.E, f);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (C > 1) {
        cluster_sync_all();  // every slice's partial sums are complete and visible
        constexpr int TPC = BM / C;        // tokens this CTA finishes
        constexpr int P = NTHREADS / TPC;  // threads per token
        const int rl = tid / P, row = slice * TPC + rl;
        if (t0 + row < p.T && !ctl->abort) {
            float* zrow = p.z + (size_t)(t0 + row) * p.E;
            const int lim = n_here < p.n_sub ? n_here : p.n_sub;
#pragma unroll 4
            for (int e = 4 * (tid - rl * P); e < lim; e += 4 * P) {
                const uint32_t a = smem_u32(part + row * ps + e);
                float4 f[C];
#pragma unroll
                for (int c = 0; c < C; ++c) f[c] = ld_cluster_f32x4(mapa_shared(a, (uint32_t)(PAIR ? 2 * c + half : c)));
                float4 z = f[0];
#pragma unroll
                for (int c = 1; c < C; ++c) {
                    z.x = __fadd_rn(z.x, f[c].x);
                    z.y = __fadd_rn(z.y, f[c].y);
                    z.z = __fadd_rn(z.z, f[c].z);
                    z.w = __fadd_rn(z.w, f[c].w);
                }
                store4(zrow, e_base + e, p.E, z);
            }
        }
    }
    // no CTA leaves while its partial sums may still be read, or while its
    // pair leader's MMAs may still read its shared memory
    if (CL > 1) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem_base, p.tmem_cols);
        else
            tmem_dealloc(tmem_base, p.tmem_cols);
    }
}

template <int C, bool PAIR>
cudaError_t launch_c(const CUtensorMap& tx, const CUtensorMap& tw, const GateParams& p, int tiles, int chunks,
                     size_t smem, cudaStream_t st) {
    constexpr auto kern = gate_logits_kernel<C, PAIR>;
    const cudaError_t err = allow_smem<kern>(SMEM_LIMIT);
    if (err != cudaSuccess) return err;
    constexpr int CL = PAIR ? 2 * C : C;
    note_launches(1);
    return launch_after(kern, dim3((unsigned)(tiles * CL), (unsigned)chunks), n_threads<PAIR>(), smem, CL, st, tx, tw, p);
}

// Clusters of `size` CTAs (1, 2, 4 or 8; one CTA per SM) resident at once on
// the current device.  Clusters stay inside a GPC, and GPCs differ in their
// SMs from chip to chip, so the runtime is asked, once per device.
int resident_clusters(int size, int num_sms) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> known[kMaxDevices][4];
    int dev = 0;
    if (size == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return num_sms / size;
    std::atomic<int>& slot = known[dev][size == 2 ? 1 : size == 4 ? 2 : 3];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    auto kern = gate_logits_kernel<2, true>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(n_threads<true>());
    cfg.dynamicSmemBytes = SMEM_LIMIT;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_LIMIT) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
        return num_sms / size * 7 / 8;
    slot.store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

cudaError_t launch_gate_logits_tc(const void* x, const void* wg, int T, int d, int E, float* logits, int* status,
                                  int num_sms, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    if (d % BK != 0 || E > kMaxExperts || E <= 0) return cudaErrorInvalidValue;
    const int n16 = (E + 15) / 16, kb = d / BK, tiles1 = (T + BM - 1) / BM;
    // CTA pairs halve the W_gate reads per token; smaller batches take the
    // one-CTA form (3000 tokens of d = 7168: 16.2 against 17.1 us, 2048: 15.0
    // against 12.9).
    const bool pair = T > 2 * BM && 8 * tiles1 > num_sms;
    const int tiles = pair ? (T + 2 * BM - 1) / (2 * BM) : tiles1;
    // K slices and chunks of experts: as many clusters as are resident at once
    // (a second wave of 8-CTA clusters took 2048 tokens from 12.9 to 26.3 us),
    // the least cost of what a CTA loads and of the partial sums it exchanges.
    // A byte of those weighs as 7 loaded (1536 tokens: 4 slices x 2 chunks 12.1
    // us, 8 x 1 16.0; 3000: 2 x 2 16.2, 4 x 1 17.9); whole sums, twice as long,
    // have to gain 5% over two halves (8192 tokens: the same time both).
    int split = 1, n_sub = n16 * 16;
    double least = 0.0;
    for (int s = pair ? 4 : 8; s >= 1; s >>= 1) {
        if (s > kb) continue;
        const int room = resident_clusters(pair ? 2 * s : s, num_sms) / tiles;
        if (room < 1 && s > 1) continue;
        const int chunks = room < 1 ? 1 : room > n16 ? n16 : room;
        const int sub = (n16 + chunks - 1) / chunks * 16;
        const double loads = (double)((kb + s - 1) / s) * (A_BYTES + (pair ? sub / 2 : sub) * BK * 2);
        const double cost = s > 1 ? loads + 7.0 * BM * sub * sizeof(float) : 1.05 * loads;
        if (least == 0.0 || cost < least) {
            least = cost;
            split = s;
            n_sub = sub;
        }
    }
    const int chunks = (n16 * 16 + n_sub - 1) / n_sub;
    GateParams p{};
    p.z = logits;
    p.T = T;
    p.E = E;
    p.n_sub = n_sub;
    p.x_rows = T < BM ? (T + 7) / 8 * 8 : BM;
    p.tmem_cols = 32;
    while (p.tmem_cols < (uint32_t)n_sub) p.tmem_cols <<= 1;  // a power of two from 32
    p.k_blocks = kb;
    p.status = status;
    const int n_rows = pair ? n_sub / 2 : n_sub;
    const int stage_bytes = A_BYTES + n_rows * BK * 2;
    const int steps = (kb + split - 1) / split;
    p.stages = (int)(RING_LIMIT / stage_bytes);
    if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
    if (p.stages > steps) p.stages = steps;
    const size_t part = split > 1 ? (size_t)BM * part_stride(n_sub) * sizeof(float) : 0;
    size_t body = (size_t)p.stages * stage_bytes;
    if (body < part) body = part;
    body = (body + 1023) / 1024 * 1024;
    p.ctl_offset = (int)body;
    size_t smem = 1024 + body + sizeof(Ctl);
    // One CTA per SM: more could ask for more TMEM than it has, and wait for it
    // while the other CTAs of their cluster hold theirs.
    if (smem < SMEM_LIMIT / 2 + 1024) smem = SMEM_LIMIT / 2 + 1024;
    if (smem > SMEM_LIMIT) return cudaErrorInvalidValue;
    CUtensorMap tx, tw;
    if (!make_tmap_2d(&tx, x, d, T, d, BK, (unsigned)p.x_rows) || !make_tmap_2d(&tw, wg, d, E, d, BK, n_rows))
        return cudaErrorInvalidValue;
    if (pair) {
        switch (split) {
            case 4: return launch_c<4, true>(tx, tw, p, tiles, chunks, smem, st);
            case 2: return launch_c<2, true>(tx, tw, p, tiles, chunks, smem, st);
            default: return launch_c<1, true>(tx, tw, p, tiles, chunks, smem, st);
        }
    }
    switch (split) {
        case 8: return launch_c<8, false>(tx, tw, p, tiles, chunks, smem, st);
        case 4: return launch_c<4, false>(tx, tw, p, tiles, chunks, smem, st);
        case 2: return launch_c<2, false>(tx, tw, p, tiles, chunks, smem, st);
        default: return launch_c<1, false>(tx, tw, p, tiles, chunks, smem, st);
    }
}

}  // namespace moe
