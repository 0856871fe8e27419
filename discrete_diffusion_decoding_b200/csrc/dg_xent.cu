// Softmax cross entropy of the vocabulary head and its gradients, in pieces of the vocabulary: no
// logits tensor is stored.
//
//   z[i, v] = h_i . W_v / T            x_i = ln sum_{v != y_i} e^{z[i, v]}
//   loss_i = ln(1 + e^{x_i - z[i, y_i]})          lse_i = z[i, y_i] + loss_i
//   G[i, v] = dloss_i / T e^{z[i, v] - lse_i}     G[i, y_i] = dloss_i / T (e^{-loss_i} - 1)
//   dh = G W        dW = G^T h
//
// The target's term is kept out of the sum: loss and the target's entry of G are then computed
// without the cancellation of lse - z[i, y_i] and of p - 1 at positions the head is sure of.
//
// Launches.  dg_xent_pack_kernel gathers the hidden states of the positions that count (target not
// ignored; backward: and dloss not 0) into a dense, zero-padded copy, so that ignored positions cost
// nothing and cannot reach a product, whatever they hold.  The number kept stays on the device; the
// products read it there.  Forward: one product over [positions, vocabulary] tiles whose epilogue
// keeps a running (maximum, sum) per row and tile, and a merge.  Backward, for each piece of the
// vocabulary: the same product again with the epilogue writing G's piece in bf16 (the operand type
// of the two products that read it; each entry is off by at most 2^-9 of itself, as the output in
// bf16 is), then one launch for both gradients' tiles, dW's written once and dh's added in fp32 to
// slabs that the last launch sums, rounds and scatters.
//
// The products run on CTA pairs (cta_group::2 UMMA, 256 x 256 tiles, K in stages of 64): warp 0
// loads (TMA, ring of kStages x 32 KB a CTA), warp 1 issues, warps 4-7 (one TMEM lane quarter each,
// thread = row) run the epilogue of one accumulator while the other is computed.  Every wait is
// bounded, and the producers leave only once the loads they issued have landed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <mutex>
#include <utility>

#include "../../include/dg.h"
#include "dg_common.cuh"
#include "dg_host.h"
#include "dg_sm100.cuh"

namespace dg {

namespace {

constexpr int kTile = 256;                 // rows and columns of an output tile (one CTA pair)
constexpr int kK = 64;                     // contraction elements per stage
constexpr int kStages = 7;
constexpr int kOperand = 16 * 1024;        // one operand's box per CTA and stage
constexpr int kStageBytes = 2 * kOperand;
constexpr int kSmem = kStages * kStageBytes + 1024;
constexpr int kXThreads = 256;
constexpr int kEpiWarp0 = 4;
constexpr int kPackRows = 16;              // rows per CTA of the gather
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum : int {
    kErrEmpty = 401, kErrFull = 402, kErrAccFree = 403, kErrAccFull = 404, kErrDrainLoads = 405, kErrDrainMma = 406,
};

enum Mode { kModeLoss, kModeLogits, kModeGrads };

__device__ __forceinline__ float exp2_sfu(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// What the gather leaves in the workspace: the positions that count, in order.
struct Packed {
    int* err;            // device error word, then the number of positions kept
    int* count;
    int32_t* row;        // original position
    int32_t* target;     // target column, -1 when it lies outside the vocabulary
    float* lse2;         // backward: lse in log2 units
    float* coef;         // backward: dloss / T
    float* tcoef;        // backward: the target's entry of G
    __nv_bfloat16* h;    // [rounded up to 256 rows, d]
};

struct PackArgs {
    Packed out;
    const __nv_bfloat16* h;
    long long h_stride;
    const void* targets;
    int targets64;
    long long ignore;
    int n, d, vocab;
    float inv_t;
    const float* loss_in;    // backward inputs (null in the forward)
    const float* lse_in;
    const float* dloss;
    float* loss_out;         // forward: ignored positions get 0 here
    float* lse_out;
    __nv_bfloat16* dh;       // backward: positions that do not count get 0 here
};

__device__ __forceinline__ bool counts(const PackArgs& a, int i, long long& y) {
    y = a.targets64 ? static_cast<const long long*>(a.targets)[i] : static_cast<const int32_t*>(a.targets)[i];
    return y != a.ignore && (!a.dloss || a.dloss[i] != 0.f);
}

__device__ __forceinline__ void zero_row(__nv_bfloat16* dst, int d, int lane) {
    for (int c = lane * 8; c < d; c += 256) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
}

// CTA b looks at rows [16 b, 16 b + 16).  Each CTA counts the kept positions before its rows (and all of them)
// itself: N / 256 coalesced reads a thread from L2, cheaper than a scan launch before this one.
__global__ void __launch_bounds__(256) dg_xent_pack_kernel(const PackArgs a) {
    __shared__ int warp_before[8], warp_all[8];
    __shared__ int slot[kPackRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = blockIdx.x * kPackRows;
    int before = 0, all = 0;
    for (int i = tid; i < a.n; i += 256) {
        long long y;
        const int k = counts(a, i, y);
        all += k;
        before += i < r0 ? k : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) {
        warp_before[warp] = before;
        warp_all[warp] = all;
    }
    __syncthreads();
    before = all = 0;
    for (int w = 0; w < 8; ++w) {
        before += warp_before[w];
        all += warp_all[w];
    }
    if (warp == 0) {
        const int i = r0 + lane;
        long long y = 0;
        const bool k = lane < kPackRows && i < a.n && counts(a, i, y);
        const uint32_t kept = __ballot_sync(0xffffffffu, k);
        const int at = before + __popc(kept & ((1u << lane) - 1u));
        if (lane < kPackRows) slot[lane] = k ? at : -1;
        if (k) {
            const bool inside = y >= 0 && y < a.vocab;
            a.out.row[at] = i;
            a.out.target[at] = inside ? static_cast<int32_t>(y) : -1;
            if (a.dloss) {
                const float c = inside ? a.dloss[i] * a.inv_t : NAN;
                a.out.coef[at] = c;
                a.out.tcoef[at] = c * expm1f(-a.loss_in[i]);
                a.out.lse2[at] = a.lse_in[i] * kLog2e;
            }
        } else if (lane < kPackRows && i < a.n && a.loss_out) {
            a.loss_out[i] = 0.f;
            if (a.lse_out) a.lse_out[i] = 0.f;
        }
        if (blockIdx.x == 0 && lane == 0) {
            *a.out.err = 0;
            *a.out.count = all;
        }
    }
    __syncthreads();
    const bool vec = (reinterpret_cast<uintptr_t>(a.h) & 15) == 0 && (a.h_stride & 7) == 0;
    const int padded = (all + kTile - 1) / kTile * kTile;
    for (int k = warp; k < kPackRows; k += 8) {
        const int i = r0 + k;
        if (i < a.n) {
            const int s = slot[k];
            const __nv_bfloat16* src = a.h + static_cast<long long>(i) * a.h_stride;
            if (s < 0) {
                if (a.dh) zero_row(a.dh + static_cast<long long>(i) * a.d, a.d, lane);
            } else if (vec) {
                __nv_bfloat16* dst = a.out.h + static_cast<long long>(s) * a.d;
                for (int c = lane * 8; c < a.d; c += 256)
                    *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + c);
            } else {
                __nv_bfloat16* dst = a.out.h + static_cast<long long>(s) * a.d;
                for (int c = lane; c < a.d; c += 32) dst[c] = src[c];
            }
        }
        // the rows behind the last one kept, up to a whole tile
        if (i >= all && i < padded) zero_row(a.out.h + static_cast<long long>(i) * a.d, a.d, lane);
    }
}

// ------------------------------------------------------------------ the products
struct GemmArgs {
    // kModeLoss, kModeLogits: a0 = packed h, b0 = W, both K-major (boxes of 64 x 128 rows).
    // kModeGrads: a0 = G K-major and b0 = W's piece MN-major for dh; a1 = G and b1 = packed h, both
    // MN-major (boxes of 64 columns x 64 rows), for dW.
    CUtensorMap a0, b0, a1, b1;
    Packed pk;
    int vocab, d;
    int v0, v_tiles;         // the piece's first column and its tiles of 256
    int d_tiles;
    float scale_log2;        // log2(e) / T
    // kModeLoss
    float2* part;            // [row][v_tiles] (maximum, sum relative to it) in log2 units
    float* zt2;              // the target's logit, log2 units
    // kModeLogits / kModeGrads
    __nv_bfloat16* g;        // [rows][g_stride]
    int g_stride;
    // kModeGrads
    float* slab;             // [splits][slab_rows][d] fp32 sums of dh
    long long slab_stride;   // elements between slabs
    int splits, kb_per_split;
    int first_piece;
    int want_dh, want_dw;
    void* dw;
    int dw_fp32, dw_accumulate;
};

// One output tile and its contraction range, in stages.
struct Item {
    int m0, n0, kb0, kbs, split;
    bool dw;
};

template <int kMode>
__device__ __forceinline__ int item_count(const GemmArgs& a, int m_tiles) {
    if (kMode != kModeGrads) return m_tiles * a.v_tiles;
    return (a.want_dh ? m_tiles * a.d_tiles * a.splits : 0) + (a.want_dw ? a.v_tiles * a.d_tiles : 0);
}

// Neighbouring items share the larger operand's tile, so that pairs at work together read it from L2.
template <int kMode>
__device__ __forceinline__ Item item_at(const GemmArgs& a, int t, int m_tiles, int rows) {
    Item it;
    if (kMode != kModeGrads) {
        it.m0 = (t % m_tiles) * kTile;
        it.n0 = (t / m_tiles) * kTile;
        it.kb0 = 0;
        it.kbs = (a.d + kK - 1) / kK;
        it.split = 0;
        it.dw = false;
        return it;
    }
    const int n_dh = a.want_dh ? m_tiles * a.d_tiles * a.splits : 0;
    it.dw = t >= n_dh;
    if (it.dw) t -= n_dh;
    it.n0 = (t % a.d_tiles) * kTile;
    const int r = t / a.d_tiles;
    if (it.dw) {
        it.m0 = r * kTile;
        it.split = 0;
        it.kb0 = 0;
        it.kbs = (rows + kK - 1) / kK;
    } else {
        it.m0 = (r % m_tiles) * kTile;
        it.split = r / m_tiles;
        it.kb0 = it.split * a.kb_per_split;
        const int all = a.v_tiles * (kTile / kK);
        it.kbs = min(a.kb_per_split, all - it.kb0);
    }
    return it;
}

// 32 accumulator columns of this thread's row, by the whole warp together.
__device__ __forceinline__ void acc_ld32(uint32_t addr, uint32_t (&r)[32]) {
    __syncwarp();
    tmem_ld32(addr, r);
    tmem_wait_ld();
}

__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// This row's logits tile -> running maximum and sum over the columns other than the target.
__device__ __forceinline__ void loss_epilogue(const GemmArgs& a, const Item& it, uint32_t acc, int i, int rows) {
    const int tgt = i < rows ? a.pk.target[i] : -1;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 32) {
        uint32_t r[32];
        acc_ld32(acc + c0, r);
        const int col = it.n0 + c0;
        float z[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) z[k] = __uint_as_float(r[k]) * a.scale_log2;
        if (col + 32 > a.vocab) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (col + k >= a.vocab) z[k] = -INFINITY;
        }
        const int off = tgt - col;
        if (off >= 0 && off < 32) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (k == off) {
                    a.zt2[i] = z[k];
                    z[k] = -INFINITY;
                }
        }
        float top = z[0];
#pragma unroll
        for (int k = 1; k < 32; ++k) top = fmaxf(top, z[k]);
        const float m2 = fmaxf(m, top);
        const float ref = m2 == -INFINITY ? 0.f : m2;     // nothing but masked columns so far
        l *= exp2_sfu(m - ref);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            s0 += exp2_sfu(z[k] - ref);
            s1 += exp2_sfu(z[k + 1] - ref);
        }
        l += s0 + s1;
        m = m2;
    }
    if (i < rows)
        a.part[static_cast<long long>(i) * a.v_tiles + it.n0 / kTile] = make_float2(m, l);
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// This row's logits tile -> its entries of G in bf16; rows and columns outside are 0.
__device__ __forceinline__ void logits_epilogue(const GemmArgs& a, const Item& it, uint32_t acc, int i, int rows) {
    const bool live = i < rows;
    const int tgt = live ? a.pk.target[i] - a.v0 : -1;
    const float coef = live ? a.pk.coef[i] : 0.f, tcoef = live ? a.pk.tcoef[i] : 0.f;
    const float lse2 = live ? a.pk.lse2[i] : 0.f;
    __nv_bfloat16* out = a.g + static_cast<long long>(i) * a.g_stride + it.n0;
    const int limit = a.vocab - a.v0;
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 32) {
        uint32_t r[32];
        acc_ld32(acc + c0, r);
        const int col = it.n0 + c0;
        float g[32];
#pragma unroll
        for (int k = 0; k < 32; ++k)
            g[k] = live ? exp2_sfu(fmaf(__uint_as_float(r[k]), a.scale_log2, -lse2)) * coef : 0.f;
        const int off = tgt - col;
        if (off >= 0 && off < 32) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (k == off) g[k] = tcoef;
        }
        if (col + 32 > limit) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (col + k >= limit) g[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
            uint32_t u[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) u[q] = bf16_pair(g[k + 2 * q], g[k + 2 * q + 1]);
            store32(out + c0 + k, u);
        }
    }
}

// A dh tile: added to (first piece: stored in) the split's fp32 slab.  Each address is touched by one
// thread of one launch at a time, so the order of the sums is that of the pieces.
__device__ __forceinline__ void dh_epilogue(const GemmArgs& a, const Item& it, uint32_t acc, int i, int rows) {
    float* out = a.slab + it.split * a.slab_stride + static_cast<long long>(i) * a.d + it.n0;
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 32) {
        uint32_t r[32];
        acc_ld32(acc + c0, r);
        if (i < rows) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                if (it.n0 + c0 + k >= a.d) break;
                if (a.first_piece)
                    *reinterpret_cast<uint4*>(out + c0 + k) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                else
                    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(out + c0 + k),
                                 "f"(__uint_as_float(r[k])), "f"(__uint_as_float(r[k + 1])),
                                 "f"(__uint_as_float(r[k + 2])), "f"(__uint_as_float(r[k + 3]))
                                 : "memory");
            }
        }
    }
}

// A dW tile: stored, or added to what is there.  `empty`: no position counts, the sum is 0.
__device__ __forceinline__ void dw_epilogue(const GemmArgs& a, const Item& it, uint32_t acc, int row, bool empty) {
    const long long v = static_cast<long long>(a.v0) + it.m0 + row;
    const bool live = v < a.vocab;
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 32) {
        uint32_t r[32];
        acc_ld32(acc + c0, r);
        if (!live) continue;
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = empty ? 0.f : __uint_as_float(r[k]);
        const long long at = v * a.d + it.n0 + c0;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
            if (it.n0 + c0 + k >= a.d) break;
            if (a.dw_fp32) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at + k);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float4 y = make_float4(x[k + 4 * q], x[k + 4 * q + 1], x[k + 4 * q + 2], x[k + 4 * q + 3]);
                    if (a.dw_accumulate) {
                        const float4 o = p[q];
                        y = make_float4(y.x + o.x, y.y + o.y, y.z + o.z, y.w + o.w);
                    }
                    p[q] = y;
                }
            } else {
                uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dw) + at + k);
                if (a.dw_accumulate) {
                    const uint4 o = *p;
                    const uint32_t u[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x[k + 2 * q] += __uint_as_float(u[q] << 16);
                        x[k + 2 * q + 1] += __uint_as_float(u[q] & 0xFFFF0000u);
                    }
                }
                *p = make_uint4(bf16_pair(x[k], x[k + 1]), bf16_pair(x[k + 2], x[k + 3]),
                                bf16_pair(x[k + 4], x[k + 5]), bf16_pair(x[k + 6], x[k + 7]));
            }
        }
    }
}

template <int kMode>
__global__ void __launch_bounds__(kXThreads, 1) dg_xent_gemm_kernel(const __grid_constant__ GemmArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // full: the leader's, counting both CTAs' bytes; acc_full / acc_free: the two accumulators
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_free[2], drain_bar, peer_bar;
    __shared__ uint32_t tmem_base, peer_issued;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t prank = cluster_ctarank();
    const bool leader = prank == 0;
    int* err = a.pk.err;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 2);          // leader: the epilogues of both CTAs
        }
        mbar_init(&drain_bar, 1);
        mbar_init(&peer_bar, 1);
        fence_mbar_init_cluster();
        abort_flag = 0;
    }
    if (warp == 1) {
        tmem_alloc_pair(&tmem_base, 2 * kTile);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    griddep_wait();          // everything read below was written by the launches before this one
    fence_async_global();    // and some of it is read by TMA

    const uint32_t tmem = tmem_base;
    const int rows = *a.pk.count;
    const int m_tiles = (rows + kTile - 1) / kTile;
    const int items = item_count<kMode>(a, m_tiles);
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t issued = 0;
            bool ok = true;
            for (int t = pair; t < items && ok; t += pairs) {
                const Item it = item_at<kMode>(a, t, m_tiles, rows);
                const CUtensorMap* ma = kMode == kModeGrads && it.dw ? &a.a1 : &a.a0;
                const CUtensorMap* mb = kMode == kModeGrads && it.dw ? &a.b1 : &a.b0;
                const int m = it.m0 + static_cast<int>(prank) * 128, n = it.n0 + static_cast<int>(prank) * 128;
                for (int kb = it.kb0; kb < it.kb0 + it.kbs; ++kb) {
                    const int s = issued % kStages;
                    if (issued >= kStages &&
                        !mbar_wait(&empty[s], ((issued / kStages) - 1) & 1, &abort_flag, err, kErrEmpty)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = ring + s * kStageBytes;
                    uint8_t* sb = sa + kOperand;
                    ++issued;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2u * kStageBytes);
                    const uint32_t bar = smem_addr_in_rank(&full[s], 0);
                    if (kMode == kModeGrads && it.dw) {
                        tma_load_2d_pair(sa, ma, bar, m, kb * kK);
                        tma_load_2d_pair(sa + kOperand / 2, ma, bar, m + 64, kb * kK);
                    } else {
                        tma_load_2d_pair(sa, ma, bar, kb * kK, m);
                    }
                    if (kMode == kModeGrads) {
                        tma_load_2d_pair(sb, mb, bar, n, kb * kK);
                        tma_load_2d_pair(sb + kOperand / 2, mb, bar, n + 64, kb * kK);
                    } else {
                        tma_load_2d_pair(sb, mb, bar, kb * kK, n);
                    }
                }
            }
            // Leave only once every load issued into either CTA has landed.  Both CTAs issue the same
            // sequence of stages, all counted on the leader's barriers; after an abort the counts of a
            // slot differ by at most one use (the next use of a slot waits for the other CTA's bytes of
            // this one), which the leader settles with the bytes that will not come.
            if (!leader) {
                st_shared_rank_u32(&peer_issued, 0, issued);
                mbar_arrive_remote(&peer_bar, 0);
            } else {
                const uint64_t t0 = global_ns();
                auto wait = [&](uint64_t* bar, uint32_t parity, bool cluster) {
                    while (!(cluster ? mbar_try_wait_cluster(smem_u32(bar), parity)
                                     : mbar_try_wait(smem_u32(bar), parity)))
                        if (global_ns() - t0 > 2 * DG_WAIT_LIMIT_NS) {
                            atomicCAS(err, 0, kErrDrainLoads);
                            return false;
                        }
                    return true;
                };
                if (wait(&peer_bar, 0, true)) {
                    const uint32_t theirs = peer_issued;
                    for (uint32_t s = 0; s < kStages; ++s) {
                        // uses of slot s: s, s + kStages, ...
                        const uint32_t mine_n = issued > s ? (issued - s - 1) / kStages + 1 : 0;
                        const uint32_t their_n = theirs > s ? (theirs - s - 1) / kStages + 1 : 0;
                        if (mine_n == 0 && their_n == 0) continue;
                        if (mine_n > their_n) mbar_complete_tx(&full[s], kStageBytes);
                        if (their_n > mine_n) mbar_arrive_expect_tx(&full[s], kStageBytes);
                        const uint32_t uses = mine_n > their_n ? mine_n : their_n;
                        if (!wait(&full[s], (uses - 1) & 1, false)) break;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            uint32_t used = 0;
            int n = 0;
            bool ok = true;
            for (int t = pair; t < items && ok; t += pairs, ++n) {
                const Item it = item_at<kMode>(a, t, m_tiles, rows);
                const bool a_mn = kMode == kModeGrads && it.dw, b_mn = kMode == kModeGrads;
                const uint32_t idesc = idesc_bf16_f32(kTile, kTile, a_mn, b_mn);
                const uint32_t buf = n & 1;
                if (n >= 2 && !mbar_wait(&acc_free[buf], ((n >> 1) - 1) & 1, &abort_flag, err, kErrAccFree)) break;
                tc_fence_after();
                for (int kb = 0; kb < it.kbs; ++kb) {
                    const int s = used % kStages;
                    if (!mbar_wait(&full[s], (used / kStages) & 1, &abort_flag, err, kErrFull)) {
                        ok = false;
                        break;
                    }
                    ++used;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring + s * kStageBytes), sb = sa + kOperand;
#pragma unroll
                    for (int kk = 0; kk < kK / 16; ++kk) {
                        // K-major: 32 bytes along the swizzled row; MN-major: 16 rows of 128 bytes, the two
                        // 64-column atoms half an operand apart
                        const uint64_t ad = a_mn ? smem_desc(sa + kk * 2048, kOperand / 2, 1024, kSwizzle128B)
                                                 : smem_desc(sa + kk * 32, 16, 1024, kSwizzle128B);
                        const uint64_t bd = b_mn ? smem_desc(sb + kk * 2048, kOperand / 2, 1024, kSwizzle128B)
                                                 : smem_desc(sb + kk * 32, 16, 1024, kSwizzle128B);
                        umma_ss_pair(tmem + buf * kTile, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
                    }
                    umma_commit_pair(&empty[s], 0x3);
                }
                if (ok) umma_commit_pair(&acc_full[buf], 0x3);
            }
            // every UMMA issued has completed before TMEM is released
            umma_commit_pair(&drain_bar, 0x1);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(smem_u32(&drain_bar), 0)) {
                if (global_ns() - t0 > DG_WAIT_LIMIT_NS) {
                    atomicCAS(err, 0, kErrDrainMma);
                    break;
                }
            }
        }
    } else if (warp >= kEpiWarp0) {
        const int row = (warp - kEpiWarp0) * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        int n = 0;
        for (int t = pair; t < items; t += pairs, ++n) {
            const Item it = item_at<kMode>(a, t, m_tiles, rows);
            const uint32_t buf = n & 1;
            mbar_wait(&acc_full[buf], (n >> 1) & 1, &abort_flag, err, kErrAccFull);
            epi_bar();
            if (abort_flag) break;
            tc_fence_after();
            const uint32_t acc = tmem + lane_addr + buf * kTile;
            const int r = it.m0 + static_cast<int>(prank) * 128 + row;
            if (kMode == kModeLoss) loss_epilogue(a, it, acc, r, rows);
            else if (kMode == kModeLogits) logits_epilogue(a, it, acc, r, rows);
            else if (it.dw) dw_epilogue(a, it, acc, static_cast<int>(prank) * 128 + row, rows == 0);
            else dh_epilogue(a, it, acc, r, rows);
            tc_fence_before();
            epi_bar();
            if (tid == kEpiWarp0 * 32) mbar_arrive_remote(&acc_free[buf], 0);
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc_pair(tmem, 2 * kTile);
}

// ------------------------------------------------------------------ merges
// One warp per kept position: the tiles' (maximum, sum) -> loss and lse.
__global__ void __launch_bounds__(256) dg_xent_merge_kernel(Packed pk, const float2* part, const float* zt2, int v_tiles,
                                                            float* loss, float* lse) {
    griddep_wait();
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= *pk.count) return;
    float m = -INFINITY, l = 0.f;
    const float2* p = part + static_cast<long long>(i) * v_tiles;
    for (int k = lane; k < v_tiles; k += 32) {
        const float2 x = p[k];
        const float m2 = fmaxf(m, x.x), ref = m2 == -INFINITY ? 0.f : m2;
        l = l * exp2f(m - ref) + x.y * exp2f(x.x - ref);
        m = m2;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, off), ol = __shfl_xor_sync(0xffffffffu, l, off);
        const float m2 = fmaxf(m, om), ref = m2 == -INFINITY ? 0.f : m2;
        l = l * exp2f(m - ref) + ol * exp2f(om - ref);
        m = m2;
    }
    if (lane == 0) {
        const int at = pk.row[i];
        float value = NAN, total = NAN;
        if (*pk.err == 0 && pk.target[i] >= 0) {
            const float zt = zt2[i];
            const float gap = l > 0.f || l != l ? (m - zt + log2f(l)) * kLn2 : -INFINITY;   // no other column: -inf
            value = fmaxf(gap, 0.f) + log1pf(expf(-fabsf(gap)));
            total = zt * kLn2 + value;
        }
        loss[at] = value;
        if (lse) lse[at] = total;
    }
}

// dh rows: the slabs' sum in bf16 at the original positions.  After a wait that ran out both gradients are NaN.
__global__ void __launch_bounds__(256) dg_xent_finish_kernel(Packed pk, const float* slab, long long slab_stride,
                                                             int splits, int d, __nv_bfloat16* dh, uint32_t* dw_words,
                                                             long long n_dw_words) {
    griddep_wait();
    const bool bad = *pk.err != 0;
    const int rows = *pk.count;
    const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    if (bad && dw_words)
        for (long long k = first; k < n_dw_words; k += step) dw_words[k] = 0x7FFF7FFFu;     // NaN as bf16 and as fp32
    if (!dh) return;
    const int vecs = d / 8;
    for (long long k = first; k < static_cast<long long>(rows) * vecs; k += step) {
        const int i = static_cast<int>(k / vecs), c = static_cast<int>(k % vecs) * 8;
        const float* src = slab + static_cast<long long>(i) * d + c;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < splits; ++s) {
            const float4 u = *reinterpret_cast<const float4*>(src + s * slab_stride);
            const float4 w = *reinterpret_cast<const float4*>(src + s * slab_stride + 4);
            x[0] += u.x;
            x[1] += u.y;
            x[2] += u.z;
            x[3] += u.w;
            x[4] += w.x;
            x[5] += w.y;
            x[6] += w.z;
            x[7] += w.w;
        }
        uint4 o = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]),
                             bf16_pair(x[6], x[7]));
        if (bad) o = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
        *reinterpret_cast<uint4*>(dh + static_cast<long long>(pk.row[i]) * d + c) = o;
    }
}

// ------------------------------------------------------------------ host side
struct XentPlan {
    int rows_alloc, v_tiles, d_tiles, pairs;
    int piece;               // columns per piece of the backward
    int splits, kb_per_split;
    size_t err, row, target, lse2, coef, tcoef, zt2, h, part, g, slab, total;
};

constexpr int kMaxRows = 1 << 22;

dg_status plan_xent(const dg_xent_params* p, bool backward, XentPlan* out) {
    if (!p || p->n < 0 || p->vocab < 1 || p->hidden < 1) return DG_EINVAL;
    if (!(p->temperature > 0.f) || !std::isfinite(p->temperature)) return DG_EINVAL;
    if (p->target_type != DG_INT32 && p->target_type != DG_INT64) return DG_EINVAL;
    if (p->dw_type != DG_BF16 && p->dw_type != DG_FP32) return DG_EINVAL;
    if (p->dw_accumulate != 0 && p->dw_accumulate != 1) return DG_EINVAL;
    if (p->h_stride != 0 && p->h_stride < p->hidden) return DG_EINVAL;
    // a TMA row starts on 16 bytes; the counts below stay in 32 bits
    if (p->hidden % 8 != 0 || p->hidden > 65536 || p->n > kMaxRows || p->vocab > (1 << 28)) return DG_EUNSUPPORTED;
    const int sms = host::device_sm_count();
    if (sms <= 1) return DG_ECUDA;
    XentPlan q{};
    q.pairs = sms / 2;
    q.rows_alloc = (p->n + kTile - 1) / kTile * kTile;
    q.v_tiles = (p->vocab + kTile - 1) / kTile;
    q.d_tiles = (p->hidden + kTile - 1) / kTile;
    const int m_tiles = q.rows_alloc / kTile;
    if (static_cast<long long>(m_tiles) * q.v_tiles > 0x7fffffffLL) return DG_EUNSUPPORTED;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    const size_t n = q.rows_alloc;
    q.err = take(8);
    q.row = take(4 * n);
    q.target = take(4 * n);
    q.lse2 = take(4 * n);
    q.coef = take(4 * n);
    q.tcoef = take(4 * n);
    q.zt2 = take(4 * n);
    q.h = take(2 * n * p->hidden);
    if (!backward) {
        q.part = take(8 * n * q.v_tiles);
    } else {
        // G's piece in at most 64 MB, so that it is read back from L2
        long long piece = (64LL << 20) / (2 * static_cast<long long>(q.rows_alloc > 0 ? q.rows_alloc : 1));
        piece = piece / kTile * kTile;
        if (piece > 16384) piece = 16384;
        if (piece < 2048) piece = 2048;
        if (piece > static_cast<long long>(q.v_tiles) * kTile) piece = static_cast<long long>(q.v_tiles) * kTile;
        q.piece = static_cast<int>(piece);
        // dh: enough tiles for every pair, split along the vocabulary
        const int kbs = q.piece / kK;
        const int tiles = m_tiles * q.d_tiles;
        int splits = tiles > 0 ? (2 * q.pairs + tiles - 1) / tiles : 1;
        if (splits > kbs / 4) splits = kbs / 4;
        if (splits < 1) splits = 1;
        q.kb_per_split = (kbs + splits - 1) / splits;
        q.splits = (kbs + q.kb_per_split - 1) / q.kb_per_split;
        q.g = take(2 * n * q.piece);
        q.slab = take(4 * n * p->hidden * q.splits);
    }
    q.total = o;
    *out = q;
    return DG_OK;
}

template <class T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

Packed packed_of(const XentPlan& q, void* ws) {
    Packed k;
    k.err = at<int>(ws, q.err);
    k.count = k.err + 1;
    k.row = at<int32_t>(ws, q.row);
    k.target = at<int32_t>(ws, q.target);
    k.lse2 = at<float>(ws, q.lse2);
    k.coef = at<float>(ws, q.coef);
    k.tcoef = at<float>(ws, q.tcoef);
    k.h = at<__nv_bfloat16>(ws, q.h);
    return k;
}

// A row-major bf16 matrix with boxes of 64 columns x box_rows rows in 128-byte swizzled rows.
bool encode_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows) {
    host::EncodeTiledFn enc = host::encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {stride * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The products' shared-memory limit, raised once per device.
bool gemm_attr_set() {
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return true;
    for (auto k : {dg_xent_gemm_kernel<kModeLoss>, dg_xent_gemm_kernel<kModeLogits>, dg_xent_gemm_kernel<kModeGrads>})
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return false;
    done[dev] = true;
    return true;
}

// A kernel that waits (griddepcontrol.wait) for the one before it on the stream: set up while that one runs.
template <class... KArgs, class... Args>
cudaError_t launch_next(void (*kern)(KArgs...), int grid, int cluster, size_t smem, cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <int kMode>
cudaError_t launch_gemm(const GemmArgs& a, long long most_items, int pairs, cudaStream_t s) {
    const int grid = 2 * static_cast<int>(most_items < pairs ? most_items : pairs);
    return launch_next(dg_xent_gemm_kernel<kMode>, grid, 2, kSmem, s, a);
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Ranges [a, a + na) and [b, b + nb) overlap.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

dg_status launch_pack(const PackArgs& in, const XentPlan& q, cudaStream_t s) {
    dg_xent_pack_kernel<<<q.rows_alloc / kPackRows, 256, 0, s>>>(in);
    return cudaGetLastError() == cudaSuccess ? DG_OK : DG_ECUDA;
}

PackArgs pack_args(const dg_xent_params* p, const XentPlan& q, void* ws, const void* h, const void* targets) {
    PackArgs a;
    std::memset(&a, 0, sizeof(a));
    a.out = packed_of(q, ws);
    a.h = static_cast<const __nv_bfloat16*>(h);
    a.h_stride = p->h_stride ? p->h_stride : p->hidden;
    a.targets = targets;
    a.targets64 = p->target_type == DG_INT64;
    a.ignore = p->ignore_index;
    a.n = p->n;
    a.d = p->hidden;
    a.vocab = p->vocab;
    a.inv_t = static_cast<float>(1.0 / static_cast<double>(p->temperature));
    return a;
}

GemmArgs gemm_args(const dg_xent_params* p, const XentPlan& q, void* ws) {
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    a.pk = packed_of(q, ws);
    a.vocab = p->vocab;
    a.d = p->hidden;
    a.d_tiles = q.d_tiles;
    a.scale_log2 = static_cast<float>(1.4426950408889634 / static_cast<double>(p->temperature));
    return a;
}

}  // namespace

}  // namespace dg

using namespace dg;
using namespace dg::host;

extern "C" {

void dg_xent_params_default(dg_xent_params* p, int n, int vocab, int hidden) {
    if (!p) return;
    std::memset(p, 0, sizeof(*p));
    p->n = n;
    p->vocab = vocab;
    p->hidden = hidden;
    p->temperature = 1.0f;
    p->ignore_index = -100;
    p->target_type = DG_INT32;
    p->dw_type = DG_BF16;
}

size_t dg_xent_workspace_size(const dg_xent_params* p, int backward) {
    XentPlan f, b;
    if (plan_xent(p, false, &f) != DG_OK) return 0;
    if (!backward) return f.total;
    if (plan_xent(p, true, &b) != DG_OK) return 0;
    return b.total > f.total ? b.total : f.total;
}

dg_status dg_xent_forward(const dg_xent_params* p, const void* h_dev, const void* W_dev, const void* targets_dev,
                          float* loss_dev, float* lse_dev, void* workspace_dev, size_t workspace_bytes, void* stream) {
    set_last_launches(0);
    XentPlan q;
    const dg_status st = plan_xent(p, false, &q);
    if (st != DG_OK) return st;
    if (p->n == 0) return DG_OK;
    if (!h_dev || !W_dev || !targets_dev || !loss_dev || !workspace_dev) return DG_EINVAL;
    if (!aligned(h_dev, 2) || !aligned(W_dev, 16) || !aligned(targets_dev, p->target_type == DG_INT64 ? 8 : 4) ||
        !aligned(loss_dev, 4) || !aligned(lse_dev, 4) || !aligned(workspace_dev, 256))
        return DG_EINVAL;
    if (workspace_bytes < q.total) return DG_ENOMEM;
    if (!gemm_attr_set()) return DG_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    PackArgs pa = pack_args(p, q, workspace_dev, h_dev, targets_dev);
    pa.loss_out = loss_dev;
    pa.lse_out = lse_dev;
    GemmArgs ga = gemm_args(p, q, workspace_dev);
    ga.v_tiles = q.v_tiles;
    ga.part = at<float2>(workspace_dev, q.part);
    ga.zt2 = at<float>(workspace_dev, q.zt2);
    if (!encode_2d(&ga.a0, ga.pk.h, q.rows_alloc, p->hidden, p->hidden, 128) ||
        !encode_2d(&ga.b0, W_dev, p->vocab, p->hidden, p->hidden, 128))
        return DG_ECUDA;
    const dg_status sp = launch_pack(pa, q, s);
    if (sp != DG_OK) return sp;
    const long long items = static_cast<long long>(q.rows_alloc / kTile) * q.v_tiles;
    if (launch_gemm<kModeLoss>(ga, items, q.pairs, s) != cudaSuccess) return DG_ECUDA;
    if (launch_next(dg_xent_merge_kernel, (p->n + 7) / 8, 1, 0, s, ga.pk, static_cast<const float2*>(ga.part),
                    static_cast<const float*>(ga.zt2), q.v_tiles, loss_dev, lse_dev) != cudaSuccess)
        return DG_ECUDA;
    set_last_launches(3);
    return DG_OK;
}

dg_status dg_xent_backward(const dg_xent_params* p, const void* h_dev, const void* W_dev, const void* targets_dev,
                           const float* loss_dev, const float* lse_dev, const float* dloss_dev, void* dh_dev,
                           void* dW_dev, void* workspace_dev, size_t workspace_bytes, void* stream) {
    set_last_launches(0);
    XentPlan q;
    const dg_status st = plan_xent(p, true, &q);
    if (st != DG_OK) return st;
    if (!dh_dev && !dW_dev) return DG_EINVAL;
    const size_t dw_bytes = static_cast<size_t>(p->vocab) * p->hidden * (p->dw_type == DG_FP32 ? 4 : 2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!aligned(dW_dev, 16) || !aligned(dh_dev, 16)) return DG_EINVAL;
    if (p->n == 0) {
        if (dW_dev && !p->dw_accumulate && cudaMemsetAsync(dW_dev, 0, dw_bytes, s) != cudaSuccess) return DG_ECUDA;
        return DG_OK;
    }
    if (!h_dev || !W_dev || !targets_dev || !loss_dev || !lse_dev || !dloss_dev || !workspace_dev) return DG_EINVAL;
    if (!aligned(h_dev, 2) || !aligned(W_dev, 16) || !aligned(targets_dev, p->target_type == DG_INT64 ? 8 : 4) ||
        !aligned(loss_dev, 4) || !aligned(lse_dev, 4) || !aligned(dloss_dev, 4) || !aligned(workspace_dev, 256))
        return DG_EINVAL;
    const size_t w_bytes = static_cast<size_t>(p->vocab) * p->hidden * 2;
    const size_t dh_bytes = static_cast<size_t>(p->n) * p->hidden * 2;
    // the products read W after the first of its gradient's rows are written
    if (dW_dev && overlap(dW_dev, dw_bytes, W_dev, w_bytes)) return DG_EINVAL;
    const size_t h_bytes = 2 * (static_cast<size_t>(p->n - 1) * (p->h_stride ? p->h_stride : p->hidden) + p->hidden);
    if (dh_dev && (overlap(dh_dev, dh_bytes, W_dev, w_bytes) || overlap(dh_dev, dh_bytes, h_dev, h_bytes)))
        return DG_EINVAL;
    if (workspace_bytes < q.total) return DG_ENOMEM;
    if (!gemm_attr_set()) return DG_ECUDA;

    PackArgs pa = pack_args(p, q, workspace_dev, h_dev, targets_dev);
    pa.loss_in = loss_dev;
    pa.lse_in = lse_dev;
    pa.dloss = dloss_dev;
    pa.dh = static_cast<__nv_bfloat16*>(dh_dev);
    GemmArgs la = gemm_args(p, q, workspace_dev);
    la.g = at<__nv_bfloat16>(workspace_dev, q.g);
    la.g_stride = q.piece;
    if (!encode_2d(&la.a0, la.pk.h, q.rows_alloc, p->hidden, p->hidden, 128)) return DG_ECUDA;
    GemmArgs ga = la;
    ga.slab = at<float>(workspace_dev, q.slab);
    ga.slab_stride = static_cast<long long>(q.rows_alloc) * p->hidden;
    ga.splits = q.splits;
    ga.kb_per_split = q.kb_per_split;
    ga.want_dh = dh_dev != nullptr;
    ga.want_dw = dW_dev != nullptr;
    ga.dw = dW_dev;
    ga.dw_fp32 = p->dw_type == DG_FP32;
    ga.dw_accumulate = p->dw_accumulate;
    if (!encode_2d(&ga.a0, la.g, q.rows_alloc, q.piece, q.piece, 128) ||
        !encode_2d(&ga.a1, la.g, q.rows_alloc, q.piece, q.piece, 64) ||
        !encode_2d(&ga.b1, la.pk.h, q.rows_alloc, p->hidden, p->hidden, 64))
        return DG_ECUDA;
    const dg_status sp = launch_pack(pa, q, s);
    if (sp != DG_OK) return sp;
    int launches = 1;
    const int m_tiles = q.rows_alloc / kTile;
    for (int v0 = 0; v0 < p->vocab; v0 += q.piece) {
        const int cols = p->vocab - v0 < q.piece ? p->vocab - v0 : q.piece;
        la.v0 = ga.v0 = v0;
        la.v_tiles = ga.v_tiles = (cols + kTile - 1) / kTile;
        const void* W_piece = static_cast<const __nv_bfloat16*>(W_dev) + static_cast<size_t>(v0) * p->hidden;
        if (!encode_2d(&la.b0, W_piece, cols, p->hidden, p->hidden, 128) ||
            !encode_2d(&ga.b0, W_piece, cols, p->hidden, p->hidden, 64))
            return DG_ECUDA;
        ga.first_piece = v0 == 0;
        const long long items = static_cast<long long>(m_tiles) * la.v_tiles;
        if (launch_gemm<kModeLogits>(la, items, q.pairs, s) != cudaSuccess) return DG_ECUDA;
        // a short last piece may need fewer splits; those left out keep their sums
        ga.splits = (ga.v_tiles * (kTile / kK) + q.kb_per_split - 1) / q.kb_per_split;
        const long long grads = (ga.want_dh ? static_cast<long long>(m_tiles) * q.d_tiles * ga.splits : 0) +
                                (ga.want_dw ? static_cast<long long>(ga.v_tiles) * q.d_tiles : 0);
        if (launch_gemm<kModeGrads>(ga, grads, q.pairs, s) != cudaSuccess) return DG_ECUDA;
        launches += 2;
    }
    const long long work = static_cast<long long>(p->n) * (p->hidden / 8);
    long long blocks = (work + 255) / 256;
    if (blocks > q.pairs * 16LL) blocks = q.pairs * 16LL;
    if (launch_next(dg_xent_finish_kernel, static_cast<int>(blocks), 1, 0, s, ga.pk, static_cast<const float*>(ga.slab),
                    ga.slab_stride, q.splits, p->hidden, static_cast<__nv_bfloat16*>(dh_dev),
                    static_cast<uint32_t*>(dW_dev), static_cast<long long>(dw_bytes / 4)) != cudaSuccess)
        return DG_ECUDA;
    set_last_launches(launches + 1);
    return DG_OK;
}

}  // extern "C"
