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
// ignored; backward: and dloss not 0) into a dense copy, so that ignored positions cost nothing and
// cannot reach a product, whatever they hold.  The number kept stays on the device; the products
// read it there.  It also takes the target's logit, as one fp32 dot product: the largest term of the
// loss is then not subject to the tensor core's truncation.  Forward: one product over [positions,
// vocabulary] tiles whose epilogue keeps a (maximum, sum) per row and half tile, and a merge.
// Backward: launch k computes G for piece k + 1 of the vocabulary (the same product, G written in
// bf16, the operand type of the two products that read it: each entry is off by at most 2^-8 of
// itself, as an output in bf16 is; see kRestList for the target's) and both gradients' tiles for
// piece k, so that the tails, the memory-bound and the compute-bound tiles of the three overlap; dW
// is written once, but for its targets' rows, and dh is added in fp32 to slabs that the last launch
// sums, rounds and scatters.
//
// The products run on CTA pairs (cta_group::2 UMMA, 256 x 256 tiles, K in stages of 64).  An item is two
// tiles side by side that share A: 48 KB a stage and CTA for 1024 tensor cycles, where one tile takes 32 KB for
// 512 and the reads from L2 (about 50 bytes a cycle and SM here) hold the tensor core at 0.78.  Warp 0 loads
// (TMA, a ring of 12 boxes), warp 1 issues, warp 2 of the pair's leader fetches items from a counter in memory
// (longest kind first, single tiles last, so that the pairs finish together), warps 4-11 (two for each TMEM lane
// quarter, each one half of a tile's columns, thread = row) take the two accumulators in turn to registers and
// run the epilogue there; the next item's first stages are multiplied for the first accumulator meanwhile.
// Every wait is bounded, and the producers leave only once the loads they issued have landed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <utility>

#include "../../include/dg.h"
#include "dg_common.cuh"
#include "dg_host.h"
#include "dg_sm100.cuh"

namespace dg {

namespace {

constexpr int kTile = 256;                 // rows and columns of an output tile (one CTA pair)
constexpr int kHalf = kTile / 2;           // rows of a CTA, columns of an epilogue group
constexpr int kK = 64;                     // contraction elements per stage
constexpr int kOperand = 16 * 1024;        // one 128 x 64 operand box per CTA and stage
constexpr int kMaxStages = 6;              // a stage is A and B of one or two tiles: 2 or 3 of the ring's boxes
constexpr int kBoxes = 12;
constexpr int kXThreads = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiBytes = 4096;            // an epilogue warp's rows on their way out: 32 x 128 bytes
constexpr int kSmemBytes = kBoxes * kOperand + 8 * kEpiBytes + 1024;
constexpr int kSched = 2;                  // items in hand: the one in work and the next
constexpr int kPackRows = 8;               // rows a CTA of the gather looks at together
// The target's entry is most of a row of G, and its rounding to bf16 would move all of dh and of that row of dW
// together.  The last launch adds what it leaves out, in fp32: to dh the remainder times the target's row of W, and to
// the rows of dW that are a target's the remainders times their positions' hidden states.  The products keep those
// rows of dW unrounded beside it for that (Packed::dw_rows; Packed::first_of tells them, from the launch before the
// first of dW).  The gradients are then as far from the 64-bit result as their own type's rounding, 0.0017 of their
// norm instead of 0.0024, for 0.5 us more at 256 positions, V = 4096, d = 128 (backward 27.6 us) and at most 1 % of the
// larger ones.  (A search through the targets by each item's epilogue instead of first_of: 5 % at 256 positions of
// V = 262144.  One CTA for a target instead of one for each part of its row: 15.2 instead of 14.2 ms where all of
// 4096 positions have one.)
constexpr int kNoPosition = 0x7fffffff;
constexpr int kRestScan = 2048;            // targets that a CTA looks at together there
constexpr int kRestList = 2 * kRestScan;   // positions of one target in hand there
constexpr int kRestCols = 256;             // columns of a part of a row there, where many positions have one target

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum : int {
    kErrEmpty = 401, kErrFull = 402, kErrAccFree = 403, kErrAccFull = 404, kErrDrainLoads = 405, kErrDrainMma = 406,
    kErrSchedFree = 407, kErrSched = 408,
};

// What a tile is of: the forward's logits, G's piece, dh, dW.
enum Kind { kLoss, kLogits, kDh, kDw };

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
    float* zt2;          // forward: the target's logit in log2 units
    float* lse2;         // backward: lse in log2 units
    float* coef;         // backward: dloss / T
    float* tcoef;        // backward: the target's entry of G
    float* trest;        // and what its rounding to bf16 leaves out
    int32_t* first_of;   // backward, dW: [vocab] the first position of each row of W that is a target, or kNoPosition
    float* dw_rows;      // backward: dW's rows of targets before their rounding, of target y with first position i in
    int dw_by_position;  // row i of [n, d] where there are fewer positions than rows of W, else in row y of [vocab, d]
    __nv_bfloat16* h;    // [rounded up to 256 rows, d]; zeros up to a multiple of 64 rows
    uint32_t* tickets;   // one counter of items for each launch of products
    int n_tickets;
};

struct PackArgs {
    Packed out;
    const __nv_bfloat16* h;
    const __nv_bfloat16* W;
    long long h_stride;
    const void* targets;
    int targets64;
    long long ignore;
    int n, d, vocab;
    int rows_per_cta;        // a multiple of 8
    int row_ctas;            // the CTAs behind these clear first_of,
    int clears;              // so many at most (0: it is not used)
    float inv_t, scale_log2;
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

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), acc);
        acc = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), acc);
    }
    return acc;
}

// A CTA looks at rows_per_cta rows, 8 at a time, a warp at one.  Each CTA counts the kept positions before its
// rows (and all of them) itself: N / 256 coalesced reads a thread from L2, cheaper than a scan launch before this
// one (8 rows a CTA up to 16384 positions; more rows for more, so that these reads stay linear in N).
__global__ void __launch_bounds__(256) dg_xent_pack_kernel(const PackArgs a) {
    __shared__ int warp_before[8], warp_all[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = blockIdx.x * a.rows_per_cta;
    griddep_launch();
    griddep_wait();
    if (static_cast<int>(blockIdx.x) >= a.row_ctas) {
        const int step = (static_cast<int>(gridDim.x) - a.row_ctas) * 256;
        for (int v = (static_cast<int>(blockIdx.x) - a.row_ctas) * 256 + tid; v < a.vocab; v += step)
            a.out.first_of[v] = kNoPosition;
        return;
    }
    int before = 0, all = 0;
#pragma unroll 4
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
    if (blockIdx.x == 0) {
        if (tid == 0) {
            *a.out.err = 0;
            *a.out.count = all;
        }
        for (int i = tid; i < a.out.n_tickets; i += 256) a.out.tickets[i] = 0;
    }
    const bool vec = (reinterpret_cast<uintptr_t>(a.h) & 15) == 0 && (a.h_stride & 7) == 0;
    for (int r = r0; r < r0 + a.rows_per_cta; r += kPackRows) {
        // lanes 0..7 look at these rows; every warp does, for its own row's place
        long long y = 0;
        const bool k = lane < kPackRows && r + lane < a.n && counts(a, r + lane, y);
        const uint32_t kept = __ballot_sync(0xffffffffu, k);
        const int i = r + warp, at = before + __popc(kept & ((1u << warp) - 1u));
        before += __popc(kept);
        y = __shfl_sync(0xffffffffu, y, warp);
        // the rows behind the last one kept, up to a whole stage of the products that sum over positions
        if (i >= all && i < (all + kK - 1) / kK * kK) zero_row(a.out.h + static_cast<long long>(i) * a.d, a.d, lane);
        if (i >= a.n) continue;
        if (!(kept >> warp & 1u)) {
            if (lane == 0 && a.loss_out) {
                a.loss_out[i] = 0.f;
                if (a.lse_out) a.lse_out[i] = 0.f;
            }
            if (a.dh) zero_row(a.dh + static_cast<long long>(i) * a.d, a.d, lane);
            continue;
        }
        const bool inside = y >= 0 && y < a.vocab;
        const __nv_bfloat16* src = a.h + static_cast<long long>(i) * a.h_stride;
        __nv_bfloat16* dst = a.out.h + static_cast<long long>(at) * a.d;
        if (vec) {
#pragma unroll 4
            for (int c = lane * 8; c < a.d; c += 256)
                *reinterpret_cast<uint4*>(dst + c) = __ldg(reinterpret_cast<const uint4*>(src + c));
        } else {
#pragma unroll 4
            for (int c = lane; c < a.d; c += 32) dst[c] = __ldg(src + c);
        }
        float zt = 0.f;
        if (!a.dloss && inside) {
            // read back what this warp has just written: the same values, whatever h's alignment
            __syncwarp();
            const __nv_bfloat16* w = a.W + y * a.d;
#pragma unroll 4
            for (int c = lane * 8; c < a.d; c += 256)
                zt = dot8(*reinterpret_cast<const uint4*>(dst + c), __ldg(reinterpret_cast<const uint4*>(w + c)), zt);
#pragma unroll
            for (int off = 16; off; off >>= 1) zt += __shfl_xor_sync(0xffffffffu, zt, off);
        }
        if (lane == 0) {
            a.out.row[at] = i;
            a.out.target[at] = inside ? static_cast<int32_t>(y) : -1;
            if (a.dloss) {
                const float c = inside ? a.dloss[i] * a.inv_t : NAN;
                const float t = c * expm1f(-a.loss_in[i]);
                a.out.coef[at] = c;
                a.out.tcoef[at] = t;
                a.out.trest[at] = t - __bfloat162float(__float2bfloat16_rn(t));
                a.out.lse2[at] = a.lse_in[i] * kLog2e;
            } else {
                a.out.zt2[at] = zt * a.scale_log2;
            }
        }
    }
}

// ------------------------------------------------------------------ the products
struct GemmArgs {
    // operands, boxes of 64 columns x 128 rows (K-major) or x 64 rows (MN-major)
    CUtensorMap h_k, w_k;            // packed h (n rows: those behind are zeros that nothing reads) and W, K-major: logits
    CUtensorMap g_k, w_mn;           // G K-major, W MN-major: dh
    CUtensorMap g_mn, h_mn;          // G and packed h, MN-major: dW
    CUtensorMap g_out, dw_out;       // G and a bf16 dW as outputs, boxes of 64 columns x 32 rows
    Packed pk;
    unsigned long long wait_ns;      // limit of each wait but those of the drains
    uint32_t* ticket;                // this launch's counter
    int vocab, d, d_tiles;
    float scale_log2;                // log2(e) / T
    float2* part;                    // forward: [row][2 v_tiles] (maximum, sum relative to it), log2 units
    // backward: G's buffers (buffer b starts at row b g_rows of the maps), the piece to compute G for and the
    // piece whose gradients are computed (first column, tiles; 0 tiles: none), and the order of the kinds
    int g_rows, g_write, g_read;
    int v0_logits, tiles_logits, v0_grads, tiles_grads;
    int slab_rows, splits, kb_per_split;
    int order[3];
    int wide;                        // a kind of at least so many tiles goes in twos
    int tail;                        // but about so many of the last kind's
    int first_piece, want_dh, want_dw;
    float* slab;                     // [splits][slab_rows][d] fp32 sums of dh
    void* dw;
    int dw_fp32, dw_accumulate;
    int mark;                        // enter the targets' first positions in Packed::first_of
};

// One or two output tiles (256 rows from m0, 256 or 512 columns from n0 of its matrices) and its contraction
// range in stages.
struct Item {
    int kind, m0, n0, tiles, kb0, kbs, split;
};
constexpr int kItemWords = sizeof(Item) / 4;

// Items of a grid of `outer` x `across` tiles: two tiles side by side each, a single one where `across` is odd,
// and singles only in the last `singles` outer rows.
struct Grid {
    int outer, across, pairs_of, wide_rows;
    __device__ __forceinline__ Grid(int outer_, int across_, int singles)
        : outer(outer_), across(across_), pairs_of((across_ + 1) >> 1), wide_rows(max(0, outer_ - singles)) {}
    __device__ __forceinline__ int count() const { return wide_rows * pairs_of + (outer - wide_rows) * across; }
    // item t -> its outer row, first tile and number of tiles
    __device__ __forceinline__ void at(int t, int& row, int& first, int& tiles) const {
        const int wide = wide_rows * pairs_of;
        if (t < wide) {
            row = t / pairs_of;
            first = (t - row * pairs_of) * 2;
            tiles = min(2, across - first);
        } else {
            t -= wide;
            row = wide_rows + t / across;
            first = t - (t / across) * across;
            tiles = 1;
        }
    }
};

// Item t of the launch.  Neighbouring items share rows of the larger operand, so that pairs at work together read
// them from L2.  false behind the last item.
template <bool kForward>
__device__ __forceinline__ bool item_at(const GemmArgs& a, int t, int m_tiles, int rows, Item& it) {
    if (t < 0) return false;
    it.kb0 = it.split = 0;
    const int kinds = kForward ? 1 : 3;
#pragma unroll
    for (int k = 0; k < kinds; ++k) {
        it.kind = kForward ? static_cast<int>(kLoss) : a.order[k];
        const int tail = k == kinds - 1 ? a.tail : 0;
        if (kForward || it.kind == kLogits) {
            // vocabulary tiles in twos, each with every tile of positions in turn; the last ones one by one
            const int singles = m_tiles * a.tiles_logits < a.wide
                                    ? a.tiles_logits
                                    : min(a.tiles_logits, (tail + m_tiles - 1) / max(m_tiles, 1));
            const int twos = (a.tiles_logits - singles) >> 1;
            const int count = (a.tiles_logits - twos) * m_tiles;
            if (t < count) {
                const int c = t / m_tiles;
                it.m0 = (t - c * m_tiles) * kTile;
                it.tiles = c < twos ? 2 : 1;
                it.n0 = (c < twos ? 2 * c : twos + c) * kTile;
                it.kbs = (a.d + kK - 1) / kK;
                return true;
            }
            t -= count;
        } else {
            const bool dw = it.kind == kDw;
            const int outer = dw ? (a.want_dw ? a.tiles_grads : 0)
                                 : (a.want_dh && a.tiles_grads ? m_tiles * a.splits : 0);
            const Grid g(outer, a.d_tiles, outer * a.d_tiles < (dw ? a.wide : a.wide / 2) ? outer : (tail + a.d_tiles - 1) / a.d_tiles);
            if (t < g.count()) {
                int r, c;
                g.at(t, r, c, it.tiles);
                it.n0 = c * kTile;
                if (dw) {
                    it.m0 = r * kTile;
                    it.kbs = (rows + kK - 1) / kK;
                } else {
                    it.split = r / m_tiles;
                    it.m0 = (r - it.split * m_tiles) * kTile;
                    it.kb0 = it.split * a.kb_per_split;
                    it.kbs = min(a.kb_per_split, a.tiles_grads * (kTile / kK) - it.kb0);
                }
                return true;
            }
            t -= g.count();
        }
    }
    return false;
}

// This thread's row of half a tile, 128 accumulator columns, by the whole warp together.  All of it goes to
// registers, so that the accumulator is free again before the epilogue begins.
__device__ __forceinline__ void acc_ld128(uint32_t addr, uint32_t (&r)[kHalf]) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kHalf; c += 32) tmem_ld32(addr + c, *reinterpret_cast<uint32_t(*)[32]>(&r[c]));
    tmem_wait_ld();
}

// Barrier of one epilogue group (128 threads); whether any of them says so, the same answer for all.
__device__ __forceinline__ bool group_any(int group, bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(mine)), "r"(1 + group)
        : "memory");
    return any != 0;
}

__device__ __forceinline__ void group_bar(int group) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory"); }

// A warp's 32 rows x 128 bytes go through shared memory, written by rows (thread = row): bf16 ones leave by TMA,
// fp32 ones are read back as 4 rows of 8 lanes x 16 bytes, so that an access to global memory covers whole lines
// (with 16 bytes of 32 rows a time, dh's tiles took 8 us and dW's 2.9).  Chunk c of row r lies at c ^ (r % 8): no bank conflicts either way.
__device__ __forceinline__ void row_chunk(uint32_t own, int row, int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(own + row * 128 + ((chunk ^ (row & 7)) << 4)), "r"(a),
                 "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 line_chunk(uint32_t own, int row, int chunk) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(own + row * 128 + ((chunk ^ (row & 7)) << 4))
                 : "memory");
    return v;
}

// Shared memory -> a box of an output map; completion by bulk groups.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 64 bf16 columns of the warp's rows as one box of `map` that starts inside at column x, row y (the copy clips it
// to the matrix).  `value` takes the place of this thread's column `at` where that is one of the 64.
__device__ __forceinline__ void rows_bf16(uint32_t own, int lane, const uint32_t* r, const CUtensorMap* map, int x, int y,
                                          int at = -1, float value = 0.f) {
    uint32_t u[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) u[k] = bf16_pair(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
    if (lane == 0) bulk_wait_read();          // the copy before this one has read the rows
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) row_chunk(own, lane, c, u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
    if (at >= 0 && at < 64)
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(own + lane * 128 + (((at >> 3) ^ (lane & 7)) << 4) + (at & 7) * 2),
                     "h"(static_cast<unsigned short>(bf16_pair(value, 0.f)))
                     : "memory");
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, own, x, y);
        bulk_commit();
    }
}

// 32 fp32 columns (r[at], ...) of the warp's rows, each 4 given to put(row, first column, values).
template <class Put>
__device__ __forceinline__ void rows_fp32(uint32_t own, int lane, const uint32_t* r, int rows_left, int cols_left, Put put) {
    if (lane == 0) bulk_wait_read();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c) row_chunk(own, lane, c, r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
    __syncwarp();
    const int c = lane & 7;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int row = 4 * q + (lane >> 3);
        if (row < rows_left && c * 4 < cols_left) {
            const uint4 v = line_chunk(own, row, c);
            put(row, c * 4, make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                        __uint_as_float(v.w)));
        }
    }
}

// This row's half tile of logits -> maximum and sum over the columns other than the target.
__device__ __forceinline__ void loss_epilogue(const GemmArgs& a, int n0, uint32_t (&r)[kHalf], int i, int rows) {
    if (i >= rows) return;
    const int off = a.pk.target[i] - n0;
    if (n0 + kHalf > a.vocab || (off >= 0 && off < kHalf)) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            if (k == off || n0 + k >= a.vocab) r[k] = 0xFF800000u;      // -inf
    }
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = __uint_as_float(r[k]);
#pragma unroll
    for (int k = 4; k < kHalf; ++k) t[k & 3] = fmaxf(t[k & 3], __uint_as_float(r[k]));
    const float m = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * a.scale_log2;
    const float ref = m == -INFINITY ? 0.f : m;     // nothing but masked columns
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kHalf; ++k) s[k & 3] += exp2_sfu(fmaf(__uint_as_float(r[k]), a.scale_log2, -ref));
    a.part[(static_cast<long long>(i) * a.tiles_logits) * 2 + n0 / kHalf] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
}

// This row's half tile of logits -> its entries of G in bf16; rows and columns outside are 0.
__device__ __forceinline__ void logits_epilogue(const GemmArgs& a, int n0, uint32_t (&r)[kHalf], int i, int rows,
                                                uint32_t own, int lane) {
    // rows that no later product reads (dW's sums end with the stage of the last position) are not written
    if (i - lane >= (rows + kK - 1) / kK * kK) return;
    const bool live = i < rows;
    const int limit = a.vocab - a.v0_logits;
    const float coef = live ? a.pk.coef[i] : 0.f, lse2 = live ? a.pk.lse2[i] : 0.f;
    const int off = live ? a.pk.target[i] - a.v0_logits - n0 : -1;
    if (i - lane < rows) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            r[k] = __float_as_uint(exp2_sfu(fmaf(__uint_as_float(r[k]), a.scale_log2, -lse2)) * coef);
    }
    if (!live) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k) r[k] = 0;
    }
    if (n0 + kHalf > limit) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            if (n0 + k >= limit) r[k] = 0;
    }
    const float tcoef = off >= 0 && off < kHalf ? a.pk.tcoef[i] : 0.f;
#pragma unroll
    for (int c = 0; c < kHalf; c += 64)
        rows_bf16(own, lane, &r[c], &a.g_out, n0 + c, a.g_write * a.g_rows + i - lane, off - c, tcoef);
}

// This row's half of a dh tile: added to (first piece: stored in) the split's fp32 slab.  Each address is touched
// by one thread of one launch at a time, so the order of the sums is that of the pieces.
__device__ __forceinline__ void dh_epilogue(const GemmArgs& a, int n0, int split, const uint32_t (&r)[kHalf], int i,
                                            int rows, uint32_t own, int lane) {
    float* out = a.slab + (static_cast<long long>(split) * a.slab_rows + i - lane) * a.d + n0;
    if (i - lane >= rows) return;
#pragma unroll
    for (int c = 0; c < kHalf; c += 32)
        if (n0 + c < a.d) rows_fp32(own, lane, &r[c], rows - (i - lane), a.d - (n0 + c), [&](int row, int col, const float4& x) {
            float* to = out + static_cast<long long>(row) * a.d + c + col;
            if (a.first_piece)
                *reinterpret_cast<float4*>(to) = x;
            else
                asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to), "f"(x.x), "f"(x.y), "f"(x.z),
                             "f"(x.w)
                             : "memory");
        });
}

// This row's half of a dW tile, stored or added to what is there.  `empty`: no position counts, the sum is 0.  Rows
// that are a target's (`first` is one of their positions) are kept unrounded for the last launch.
__device__ __forceinline__ void dw_epilogue(const GemmArgs& a, int n0, uint32_t (&r)[kHalf], int v, bool empty,
                                            int target_first, uint32_t own, int lane) {
    const bool of_target = target_first != kNoPosition;
    const long long first = static_cast<long long>(v - lane) * a.d + n0;
    const int rows_left = a.vocab - (v - lane);
    if (empty) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k) r[k] = 0;
    }
    if (of_target) {
        float* to = a.pk.dw_rows + static_cast<long long>(a.pk.dw_by_position ? target_first : v) * a.d + n0;
#pragma unroll
        for (int c = 0; c < kHalf; c += 4)
            if (n0 + c < a.d)
                *reinterpret_cast<float4*>(to + c) = make_float4(__uint_as_float(r[c]), __uint_as_float(r[c + 1]),
                                                                 __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, of_target);
    if (!a.dw_fp32 && !a.dw_accumulate) {
#pragma unroll
        for (int c = 0; c < kHalf; c += 64)
            if (rows_left > 0 && n0 + c < a.d) rows_bf16(own, lane, &r[c], &a.dw_out, n0 + c, v - lane);
        return;
    }
#pragma unroll
    for (int c = 0; c < kHalf; c += 32)
        if (n0 + c < a.d) rows_fp32(own, lane, &r[c], rows_left, a.d - (n0 + c), [&](int row, int col, float4 x) {
            if (kept >> row & 1u) return;
            const long long at = first + static_cast<long long>(row) * a.d + c + col;
            if (a.dw_fp32) {
                float4* to = reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at);
                if (a.dw_accumulate) {
                    const float4 o = *to;
                    x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
                }
                *to = x;
            } else {
                uint2* to = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dw) + at);
                const uint2 o = *to;
                *to = make_uint2(bf16_pair(x.x + __uint_as_float(o.x << 16), x.y + __uint_as_float(o.x & 0xFFFF0000u)),
                                 bf16_pair(x.z + __uint_as_float(o.y << 16), x.w + __uint_as_float(o.y & 0xFFFF0000u)));
            }
        });
}

template <bool kForward>
__global__ void __launch_bounds__(kXThreads, 1) dg_xent_gemm_kernel(const __grid_constant__ GemmArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // full: the leader's, counting both CTAs' bytes; acc_full / acc_free: the two accumulators;
    // sched_full / sched_free: the items fetched ahead (free: the leader's)
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_free[2], drain_bar, peer_bar;
    __shared__ uint64_t sched_full[kSched], sched_free[kSched];
    __shared__ uint32_t sched_item[kSched][kItemWords];
    __shared__ uint32_t tmem_base, peer_issued, last_bytes[kMaxStages], peer_bytes[kMaxStages];
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t prank = cluster_ctarank();
    const bool leader = prank == 0;
    int* err = a.pk.err;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 4);          // leader: two epilogue groups in each CTA
        }
        for (int i = 0; i < kSched; ++i) {
            mbar_init(&sched_full[i], 1);
            mbar_init(&sched_free[i], 7);        // leader: producers and epilogue groups of both, its issuer
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
    griddep_launch();
    if (warp == 0 && lane == 0) {
        const CUtensorMap* maps[6] = {&a.h_k, &a.w_k, &a.g_k, &a.w_mn, &a.g_mn, &a.h_mn};
#pragma unroll
        for (int i = 0; i < (kForward ? 2 : 6); ++i) tma_prefetch_desc(maps[i]);
    }
    griddep_wait();          // everything read below was written by the launches before this one
    fence_async_global();    // and some of it is read by TMA

    const uint32_t tmem = tmem_base;
    const int rows = *a.pk.count;
    const int m_tiles = (rows + kTile - 1) / kTile;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    const int m_tiles_or_dw = m_tiles + (kForward ? 0 : a.tiles_grads);
    // The n-th item of this pair: the first is its own number, the others come from the counter (false: no more, or a wait ran out).  `release`: this role is done reading it.
    auto fetch = [&](uint32_t n, Item& it) {
        if (n == 0) return m_tiles_or_dw > 0 && item_at<kForward>(a, pair, m_tiles, rows, it);
        const uint32_t s = (n - 1) % kSched;
        if (!mbar_wait<true>(&sched_full[s], ((n - 1) / kSched) & 1, &abort_flag, err, kErrSched, a.wait_ns))
            return false;
        const volatile uint32_t* w = sched_item[s];
        it = Item{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3]),
                  static_cast<int>(w[4]), static_cast<int>(w[5]), static_cast<int>(w[6])};
        return it.kind >= 0;
    };
    auto release = [&](uint32_t n) {
        if (n > 0) mbar_arrive_remote(&sched_free[(n - 1) % kSched], 0);
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t issued = 0, freed = 0, sizes = 0;     // stages; boxes of each in flight, 2 bits, newest lowest
            int head = 0, taken = 0;                       // the ring's next box, boxes in flight
            bool ok = true;
            Item it;
            for (uint32_t n = 0; ok && fetch(n, it); ++n) {
                release(n);
                const CUtensorMap *ma, *mb;
                int m = it.m0 + static_cast<int>(prank) * kHalf, c = it.n0 + static_cast<int>(prank) * kHalf;
                int ka = it.kb0 * kK, kb = ka;
                const bool a_mn = !kForward && it.kind == kDw, b_mn = !kForward && it.kind != kLogits;
                const uint32_t bytes = static_cast<uint32_t>(1 + it.tiles) * kOperand;
                if (kForward || it.kind == kLogits) {
                    ma = &a.h_k;
                    mb = &a.w_k;
                    c += kForward ? 0 : a.v0_logits;
                } else if (it.kind == kDh) {
                    ma = &a.g_k;
                    mb = &a.w_mn;
                    m += a.g_read * a.g_rows;
                    kb += a.v0_grads;
                } else {
                    ma = &a.g_mn;
                    mb = &a.h_mn;
                    ka += a.g_read * a.g_rows;
                }
                for (int k = 0; k < it.kbs; ++k, ka += kK, kb += kK) {
                    const int need = 1 + it.tiles;
                    while (taken + need > kBoxes || issued - freed >= kMaxStages) {
                        if (!mbar_wait(&empty[freed % kMaxStages], (freed / kMaxStages) & 1, &abort_flag, err,
                                       kErrEmpty, a.wait_ns)) {
                            ok = false;
                            break;
                        }
                        taken -= static_cast<int>(sizes >> (2 * (issued - freed - 1)) & 3u);
                        ++freed;
                    }
                    if (!ok) break;
                    const int s = issued % kMaxStages;
                    uint8_t* sa = ring + head * kOperand;
                    head = head + 1 == kBoxes ? 0 : head + 1;
                    taken += need;
                    sizes = sizes << 2 | static_cast<uint32_t>(need);
                    ++issued;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2u * bytes);
                    last_bytes[s] = bytes;
                    const uint32_t bar = smem_addr_in_rank(&full[s], 0);
                    if (a_mn) {
                        tma_load_2d_pair(sa, ma, bar, m, ka);
                        tma_load_2d_pair(sa + kOperand / 2, ma, bar, m + 64, ka);
                    } else {
                        tma_load_2d_pair(sa, ma, bar, ka, m);
                    }
                    for (int j = 0; j < it.tiles; ++j) {
                        const int cj = c + j * kTile;
                        uint8_t* to = ring + head * kOperand;
                        head = head + 1 == kBoxes ? 0 : head + 1;
                        if (b_mn) {
                            tma_load_2d_pair(to, mb, bar, cj, kb);
                            tma_load_2d_pair(to + kOperand / 2, mb, bar, cj + 64, kb);
                        } else {
                            tma_load_2d_pair(to, mb, bar, kb, cj);
                        }
                    }
                }
            }
            // Leave only once every load issued into either CTA has landed.  Both CTAs issue the same
            // sequence of stages, all counted on the leader's barriers; after an abort the counts of a
            // barrier differ by at most one use (the next use waits for the other CTA's bytes of this
            // one), which the leader settles with the bytes that will not come.
            if (!leader) {
                st_shared_rank_u32(&peer_issued, 0, issued);
                for (int s = 0; s < kMaxStages; ++s) st_shared_rank_u32(&peer_bytes[s], 0, last_bytes[s]);
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
                    for (uint32_t s = 0; s < kMaxStages; ++s) {
                        // uses of barrier s: s, s + kMaxStages, ...
                        const uint32_t mine_n = issued > s ? (issued - s - 1) / kMaxStages + 1 : 0;
                        const uint32_t their_n = theirs > s ? (theirs - s - 1) / kMaxStages + 1 : 0;
                        if (mine_n == 0 && their_n == 0) continue;
                        if (mine_n > their_n) mbar_complete_tx(&full[s], last_bytes[s]);
                        if (their_n > mine_n) mbar_arrive_expect_tx(&full[s], peer_bytes[s]);
                        const uint32_t uses = mine_n > their_n ? mine_n : their_n;
                        if (!wait(&full[s], (uses - 1) & 1, false)) break;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            uint32_t used = 0;              // stages
            int head = 0;                   // the ring's box of stage `used`
            uint32_t uses[2] = {0, 0};      // of the two accumulators
            int next = 0;                   // the accumulator of the next item's first tile
            bool ok = true;
            Item it;
            for (uint32_t n = 0; ok && fetch(n, it); ++n) {
                release(n);
                const bool a_mn = !kForward && it.kind == kDw, b_mn = !kForward && it.kind != kLogits;
                const uint32_t idesc = idesc_bf16_f32(kTile, kTile, a_mn, b_mn);
                // K step kk of a stage - K-major: 32 bytes along the swizzled row; MN-major: 16 rows of 128 bytes,
                // the two 64-column atoms half an operand apart
                auto box = [&](int k) { return smem_u32(ring + (k >= kBoxes ? k - kBoxes : k) * kOperand); };
                // `ahead` stages behind the current one
                auto multiply = [&](int ahead, int tile, bool accumulate) {
                    int first = head + ahead * (1 + it.tiles);
                    if (first >= kBoxes) first -= kBoxes;
                    const uint32_t sa = box(first), sb = box(first + 1 + tile);
#pragma unroll
                    for (int kk = 0; kk < kK / 16; ++kk) {
                        const uint64_t ad = a_mn ? smem_desc(sa + kk * 2048, kOperand / 2, 1024, kSwizzle128B)
                                                 : smem_desc(sa + kk * 32, 16, 1024, kSwizzle128B);
                        const uint64_t bd = b_mn ? smem_desc(sb + kk * 2048, kOperand / 2, 1024, kSwizzle128B)
                                                 : smem_desc(sb + kk * 32, 16, 1024, kSwizzle128B);
                        umma_ss_pair(tmem + (next ^ tile) * kTile, ad, bd, idesc, accumulate || kk != 0 ? 1u : 0u);
                    }
                };
                auto landed = [&](uint32_t stage) {
                    if (!mbar_wait(&full[stage % kMaxStages], (stage / kMaxStages) & 1, &abort_flag, err, kErrFull,
                                   a.wait_ns))
                        return false;
                    tc_fence_after();
                    return true;
                };
                auto acc_ready = [&](int acc) {
                    if (uses[acc] > 0 &&
                        !mbar_wait(&acc_free[acc], (uses[acc] - 1) & 1, &abort_flag, err, kErrAccFree, a.wait_ns))
                        return false;
                    ++uses[acc];
                    tc_fence_after();
                    return true;
                };
                ok = acc_ready(next);
                // the stages in the ring for the first tile, then for the second once its accumulator is free
                const int ahead = it.tiles == 2 ? min(kBoxes / 3, it.kbs) : 0;
                for (int k = 0; ok && k < ahead; ++k) {
                    ok = landed(used + k);
                    if (ok) multiply(k, 0, k != 0);
                }
                if (ok && it.tiles == 2) ok = acc_ready(next ^ 1);
                for (int k = 0; ok && k < it.kbs; ++k) {
                    if (k >= ahead) {
                        ok = landed(used);
                        if (!ok) break;
                        multiply(0, 0, k != 0);
                    }
                    if (k == it.kbs - 1) umma_commit_pair(&acc_full[next], 0x3);
                    if (it.tiles == 2) multiply(0, 1, k != 0);
                    umma_commit_pair(&empty[used % kMaxStages], 0x3);
                    ++used;
                    head += 1 + it.tiles;
                    if (head >= kBoxes) head -= kBoxes;
                }
                if (ok && it.kbs == 0) umma_commit_pair(&acc_full[next], 0x3);
                if (ok && it.tiles == 2) umma_commit_pair(&acc_full[next ^ 1], 0x3);
                if (it.tiles == 1) next ^= 1;
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
    } else if (warp == 2) {
        if (lane == 0 && leader) {
            Item it;
            bool more = fetch(0, it);
            for (uint32_t k = 0; more; ++k) {       // item k + 1
                const uint32_t s = k % kSched;
                if (k >= kSched &&
                    !mbar_wait<true>(&sched_free[s], ((k / kSched) - 1) & 1, &abort_flag, err, kErrSchedFree, a.wait_ns))
                    break;
                more = item_at<kForward>(a, pairs + static_cast<int>(atomicAdd(a.ticket, 1u)), m_tiles, rows, it);
                if (!more) it = Item{-1, 0, 0, 0, 0, 0, 0};
                const int words[kItemWords] = {it.kind, it.m0, it.n0, it.tiles, it.kb0, it.kbs, it.split};
                for (uint32_t r = 0; r < 2; ++r) {
#pragma unroll
                    for (int w = 0; w < kItemWords; ++w)
                        st_shared_rank_u32(&sched_item[s][w], r, static_cast<uint32_t>(words[w]));
                    mbar_arrive_remote(&sched_full[s], r);
                }
            }
        }
    } else if (!kForward && warp == 3) {
        // the launch before the first rows of dW: where each target stands first
        if (a.mark)
            for (int i = blockIdx.x * 32 + lane; i < rows; i += gridDim.x * 32) {
                const int y = a.pk.target[i];
                if (y >= 0) atomicMin(&a.pk.first_of[y], i);
            }
    } else if (warp >= kEpiWarp0) {
        const int group = (warp - kEpiWarp0) >> 2;                 // which half of the columns
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const bool first = tid == (kEpiWarp0 + 4 * group) * 32;
        const uint32_t own = smem_u32(ring + kBoxes * kOperand + (warp - kEpiWarp0) * kEpiBytes);
        uint32_t uses[2] = {0, 0};
        int next = 0;
        bool ok = true;
        Item it;
        for (uint32_t n = 0; ok; ++n) {
            // the same answer in every thread of the group, so that none waits alone at a barrier
            if (group_any(group, !fetch(n, it))) break;
            if (first) release(n);
            int target_first = kNoPosition;
            if (!kForward && it.kind == kDw) {
                const int v = a.v0_grads + it.m0 + static_cast<int>(prank) * kHalf + row;
                if (v < a.vocab) target_first = a.pk.first_of[v];
            }
            for (int j = 0; j < it.tiles; ++j) {
                const int buf = next ^ j;
                if (group_any(group, !mbar_wait(&acc_full[buf], uses[buf] & 1, &abort_flag, err, kErrAccFull,
                                                a.wait_ns))) {
                    ok = false;
                    break;
                }
                ++uses[buf];
                tc_fence_after();
                uint32_t r[kHalf];
                acc_ld128(tmem + lane_addr + buf * kTile + group * kHalf, r);
                tc_fence_before();
                group_bar(group);
                if (first) mbar_arrive_remote(&acc_free[buf], 0);
                const int i = it.m0 + static_cast<int>(prank) * kHalf + row;
                const int n0 = it.n0 + j * kTile + group * kHalf;
                if constexpr (kForward) {
                    loss_epilogue(a, n0, r, i, rows);
                } else {
                    if (it.kind == kLogits) logits_epilogue(a, n0, r, i, rows, own, lane);
                    else if (it.kind == kDh) dh_epilogue(a, n0, it.split, r, i, rows, own, lane);
                    else dw_epilogue(a, n0, r, a.v0_grads + i, rows == 0, target_first, own, lane);
                }
            }
            if (it.tiles == 1) next ^= 1;
        }
        if (lane == 0) bulk_wait();          // the copies out have been made
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc_pair(tmem, 2 * kTile);
}

// ------------------------------------------------------------------ few positions
// The forward's product where at most 32 positions can count: the vocabulary is the rows of the tile (128 a CTA)
// and the positions its 16 or 32 columns, so that the tensor core does not multiply 256 rows for one.  That costs
// power, and with it the clock that the reads from memory need.  Each CTA streams its rows of W through a ring of
// its own and each epilogue thread keeps a running (maximum, sum) of every position over the vocabulary rows it
// sees.  At V = 262144, d = 2816, heads in turn: 246 us for 1 position (6.0 TB/s; the kernel above 342), 248 for
// 16 (323), 254 for 32 (332).  With 64 columns the final sums over the lanes cost more than is saved on
// smaller heads (n = 64, V = 5000: 47 us against 36; n = 33, V = 50000, d = 1000: 53 against 46).
// The tensor core cuts its running sum off at every 16 products, which puts up to d / 16 units in the last place on a
// logit, all to one side.  Each sum is therefore made in kFewParts parts with an accumulator each, which the epilogue
// adds: an eighth of that (V = 262144, d = 2816, 1 position: lse off by 0.2 to 1.5e-7 of itself instead of 2 to
// 3.4e-7, in 246 us instead of 243).  The backward's logits are not made in parts, and its softmax is as far from
// adding up to 1 as they are from the forward's: past kFewPartStages one part again.  With products of one sign, logits
// of 32 and 17 positions: d = 4096 loss 1.1e-6 and dh 1.7e-3 of their norms off in parts, 3.7e-5 and 1.5e-3 in one;
// d = 8192 3.8e-6 and 3.0e-3, 1.1e-4 and 1.5e-3; d = 65536 dh 3.5e-2 and 1.5e-3.
constexpr int kFewRows = 32;               // positions at most
constexpr int kFewParts = 8;
constexpr int kFewPartStages = 64;
constexpr int kFewAcc = kFewParts * kFewRows;   // TMEM columns of a tile's accumulators, of which there are two
constexpr int kFewStages = 12;
constexpr int kFewRingBytes = 220 * 1024;
constexpr int kFewSmemBytes = kFewRingBytes + 1024;
constexpr int kFewThreads = 256;

struct FewArgs {
    CUtensorMap h, w;        // boxes of 64 columns x columns / 128 rows, K-major
    Packed pk;
    unsigned long long wait_ns;
    int vocab, d, columns;   // columns of a tile: 16 or 32
    float scale_log2;
    float2* part;            // [position][4 gridDim.x]
};

template <int kColumns>
__device__ __forceinline__ void few_epilogue(const FewArgs& a, uint32_t tmem, uint64_t* acc_full, uint64_t* acc_free,
                                             const int* target, int* abort_flag, int rows, int tiles, int parts) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127;
    float m[kColumns], l[kColumns];
#pragma unroll
    for (int c = 0; c < kColumns; ++c) {
        m[c] = -INFINITY;
        l[c] = 0.f;
    }
    int n = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
        const int buf = n & 1;
        if (group_any(0, !mbar_wait(&acc_full[buf], (n >> 1) & 1, abort_flag, a.pk.err, kErrAccFull, a.wait_ns)))
            return;
        tc_fence_after();
        const uint32_t acc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + buf * kFewAcc;
        float sum[kColumns];
#pragma unroll
        for (int c = 0; c < kColumns; ++c) sum[c] = 0.f;
        for (int part = 0; part < parts; ++part) {
            uint32_t r[kColumns];
#pragma unroll
            for (int c = 0; c < kColumns; c += 16)
                tmem_ld16(acc + part * kFewRows + c, *reinterpret_cast<uint32_t(*)[16]>(&r[c]));
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kColumns; ++c) sum[c] += __uint_as_float(r[c]);
        }
        tc_fence_before();
        group_bar(0);
        if (row == 0) mbar_arrive(&acc_free[buf]);
        const int v = t * kHalf + row;
        if (v >= a.vocab) continue;
#pragma unroll
        for (int c = 0; c < kColumns; ++c) {
            const float z = v == target[c] ? -INFINITY : sum[c] * a.scale_log2;
            const float m2 = fmaxf(m[c], z), ref = m2 == -INFINITY ? 0.f : m2;
            l[c] = l[c] * exp2_sfu(m[c] - ref) + exp2_sfu(z - ref);
            m[c] = m2;
        }
    }
#pragma unroll
    for (int c = 0; c < kColumns; ++c) {
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m[c], off), ol = __shfl_xor_sync(0xffffffffu, l[c], off);
            const float m2 = fmaxf(m[c], om), ref = m2 == -INFINITY ? 0.f : m2;
            l[c] = l[c] * exp2_sfu(m[c] - ref) + ol * exp2_sfu(om - ref);
            m[c] = m2;
        }
        if (lane == 0 && c < rows)
            a.part[(static_cast<long long>(c) * gridDim.x + blockIdx.x) * 4 + (warp & 3)] = make_float2(m[c], l[c]);
    }
}

// Launched in clusters of two for the waits' abort flags; the two CTAs share nothing else.
__global__ void __launch_bounds__(kFewThreads, 1) dg_xent_few_kernel(const __grid_constant__ FewArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kFewStages], empty[kFewStages], acc_full[2], acc_free[2], drain_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ int target[kFewRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* err = a.pk.err;
    if (tid == 0) {
        for (int i = 0; i < kFewStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 1);
        }
        mbar_init(&drain_bar, 1);
        fence_mbar_init_cluster();
        abort_flag = 0;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, 2 * kFewAcc);
        tmem_relinquish();
    }
    griddep_launch();
    if (tid == 0) {
        tma_prefetch_desc(&a.h);
        tma_prefetch_desc(&a.w);
    }
    griddep_wait();
    const int rows = *a.pk.count;
    if (tid < kFewRows) target[tid] = tid < rows ? a.pk.target[tid] : -1;
    fence_async_global();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const int tiles = rows > 0 ? (a.vocab + kHalf - 1) / kHalf : 0;
    const int kbs = (a.d + kK - 1) / kK;
    const int stage_bytes = kOperand + a.columns * 128;
    const int stages = min(kFewStages, kFewRingBytes / stage_bytes);
    const int per_part = kbs <= kFewPartStages ? (kbs + kFewParts - 1) / kFewParts : kbs;
    const int parts = (kbs + per_part - 1) / per_part;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t once = l2_policy_evict_first();
            uint32_t issued = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                for (int k = 0; k < kbs; ++k) {
                    const uint32_t s = issued % stages;
                    if (issued >= static_cast<uint32_t>(stages) &&
                        !mbar_wait(&empty[s], ((issued / stages) - 1) & 1, &abort_flag, err, kErrEmpty, a.wait_ns)) {
                        ok = false;
                        break;
                    }
                    ++issued;
                    uint8_t* to = ring + s * stage_bytes;
                    mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(stage_bytes));
                    tma_load_2d_hint(to, &a.w, &full[s], k * kK, t * kHalf, once);
                    tma_load_2d(to + kOperand, &a.h, &full[s], k * kK, 0);
                }
            }
            // leave only once every load issued has landed
            const uint64_t t0 = global_ns();
            for (uint32_t s = 0; s < static_cast<uint32_t>(stages); ++s) {
                const uint32_t uses = issued > s ? (issued - s - 1) / stages + 1 : 0;
                while (uses > 0 && !mbar_try_wait(smem_u32(&full[s]), (uses - 1) & 1))
                    if (global_ns() - t0 > DG_WAIT_LIMIT_NS) {
                        atomicCAS(err, 0, kErrDrainLoads);
                        break;
                    }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_bf16_f32(kHalf, a.columns, false, false);
            uint32_t used = 0;
            int n = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++n) {
                const int buf = n & 1;
                if (n >= 2 &&
                    !mbar_wait(&acc_free[buf], ((n >> 1) - 1) & 1, &abort_flag, err, kErrAccFree, a.wait_ns))
                    break;
                tc_fence_after();
                const uint32_t acc = tmem + buf * kFewAcc;
                for (int k = 0, part = 0, in_part = 0; k < kbs; ++k, ++used) {
                    const uint32_t s = used % stages;
                    if (!mbar_wait(&full[s], (used / stages) & 1, &abort_flag, err, kErrFull, a.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring + s * stage_bytes), sb = sa + kOperand;
#pragma unroll
                    for (int kk = 0; kk < kK / 16; ++kk)
                        umma_ss(acc + part * kFewRows, smem_desc(sa + kk * 32, 16, 1024, kSwizzle128B),
                                smem_desc(sb + kk * 32, 16, 1024, kSwizzle128B), idesc, (in_part | kk) != 0 ? 1u : 0u);
                    umma_commit(&empty[s]);
                    if (++in_part == per_part) {
                        in_part = 0;
                        ++part;
                    }
                }
                if (ok) umma_commit(&acc_full[buf]);
            }
            umma_commit(&drain_bar);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(smem_u32(&drain_bar), 0)) {
                if (global_ns() - t0 > DG_WAIT_LIMIT_NS) {
                    atomicCAS(err, 0, kErrDrainMma);
                    break;
                }
            }
        }
    } else if (warp >= 4) {
        if (a.columns == 16) few_epilogue<16>(a, tmem, acc_full, acc_free, target, &abort_flag, rows, tiles, parts);
        else few_epilogue<32>(a, tmem, acc_full, acc_free, target, &abort_flag, rows, tiles, parts);
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc(tmem, 2 * kFewAcc);
}

// ------------------------------------------------------------------ merges
__device__ __forceinline__ void merge_into(float& m, float& l, float om, float ol) {
    const float m2 = fmaxf(m, om), ref = m2 == -INFINITY ? 0.f : m2;
    l = l * exp2f(m - ref) + ol * exp2f(om - ref);
    m = m2;
}

// One CTA per kept position: the half tiles' (maximum, sum) -> loss and lse.
__global__ void __launch_bounds__(256) dg_xent_merge_kernel(Packed pk, const float2* part, int parts, float* loss,
                                                            float* lse) {
    __shared__ float2 of_warp[8];
    griddep_launch();
    griddep_wait();
    const int i = blockIdx.x, lane = threadIdx.x & 31;
    if (i >= *pk.count) return;
    float m = -INFINITY, l = 0.f;
    const float2* p = part + static_cast<long long>(i) * parts;
#pragma unroll 4
    for (int k = threadIdx.x; k < parts; k += 256) {
        const float2 x = p[k];
        merge_into(m, l, x.x, x.y);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1)
        merge_into(m, l, __shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, l, off));
    if (lane == 0) of_warp[threadIdx.x >> 5] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) merge_into(m, l, of_warp[w].x, of_warp[w].y);
        const int at = pk.row[i];
        float value = NAN, total = NAN;
        const float zt = pk.zt2[i];
        // a target's logit of +inf would make the loss 0 and its gradient vanish
        if (*pk.err == 0 && pk.target[i] >= 0 && fabsf(zt) < INFINITY) {
            const float gap = l > 0.f || l != l ? (m - zt + log2f(l)) * kLn2 : -INFINITY;   // no other column: -inf
            value = fmaxf(gap, 0.f) + log1pf(expf(-fabsf(gap)));
            total = zt * kLn2 + value;
        }
        loss[at] = value;
        if (lse) lse[at] = total;
    }
}

struct FinishArgs {
    Packed pk;
    const float* slab;
    long long slab_stride;
    int splits, d, dh_ctas;          // the first CTAs work on dh, the others on dW
    const __nv_bfloat16* W;
    __nv_bfloat16* dh;
    void* dw;
    long long dw_words;
    int dw_fp32, dw_accumulate;
};

// The remainders of `count` listed positions times their hidden states and the row's sums so far, for the columns of
// part `part` of the row, 4 a thread: the new sums, or (kLast) the row of dW.  With few positions a part is 1024
// columns; with many it is kRestCols, and the threads that share a column take the positions in turn.
template <bool kLast>
__device__ __forceinline__ void add_rest(const FinishArgs& a, float* sums, int y, const int* list, int count, bool many,
                                         int part, float4* shared) {
    const int wide = min(a.d / 4, many ? kRestCols / 4 : 256), shares = many ? 256 / wide : 1;
    const int share = threadIdx.x / wide, own = threadIdx.x - share * wide;
    const int c = (part * wide + own) * 4;
    const bool live = share < shares && c < a.d, writes = live && share == 0;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (writes) x = *reinterpret_cast<const float4*>(sums + c);
    if (live) {
        int k = share;
        auto add = [&](auto batch) {          // so many loads in flight
            constexpr int n = decltype(batch)::value;
            float t[n];
            uint2 h[n];
#pragma unroll
            for (int q = 0; q < n; ++q) {
                const int at = list[k + q * shares];
                t[q] = __ldg(a.pk.trest + at);
                h[q] = __ldg(reinterpret_cast<const uint2*>(a.pk.h + static_cast<long long>(at) * a.d + c));
            }
#pragma unroll
            for (int q = 0; q < n; ++q) {
                x.x = fmaf(t[q], __uint_as_float(h[q].x << 16), x.x);
                x.y = fmaf(t[q], __uint_as_float(h[q].x & 0xFFFF0000u), x.y);
                x.z = fmaf(t[q], __uint_as_float(h[q].y << 16), x.z);
                x.w = fmaf(t[q], __uint_as_float(h[q].y & 0xFFFF0000u), x.w);
            }
            k += n * shares;
        };
        while (k + 11 * shares < count) add(std::integral_constant<int, 12>());
        while (k + 2 * shares < count) add(std::integral_constant<int, 3>());
        while (k < count) add(std::integral_constant<int, 1>());
    }
    if (shares > 1) {
        shared[threadIdx.x] = x;
        __syncthreads();
        for (int k = 1; writes && k < shares; ++k) {
            const float4 o = shared[k * wide + own];
            x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
        }
        __syncthreads();
    }
    if (!writes) return;
    if constexpr (!kLast) {
        *reinterpret_cast<float4*>(sums + c) = x;
    } else {
        const long long to = static_cast<long long>(y) * a.d + c;
        if (a.dw_fp32) {
            float4* out = reinterpret_cast<float4*>(static_cast<float*>(a.dw) + to);
            if (a.dw_accumulate) {
                const float4 o = *out;
                x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
            }
            *out = x;
        } else {
            uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dw) + to);
            if (a.dw_accumulate) {
                const uint2 o = *out;
                x = make_float4(x.x + __uint_as_float(o.x << 16), x.y + __uint_as_float(o.x & 0xFFFF0000u),
                                x.z + __uint_as_float(o.y << 16), x.w + __uint_as_float(o.y & 0xFFFF0000u));
            }
            *out = make_uint2(bf16_pair(x.x, x.y), bf16_pair(x.z, x.w));
        }
    }
}

// dW's row of position `at`'s target, by a CTA: the remainders of all positions of that target, listed in their order.
// The row's parts go round among the CTAs of the target's first positions.  One barrier for each kRestScan targets;
// `turn` alternates the words that the warps exchange.
__device__ __forceinline__ void finish_dw_row(const FinishArgs& a, int at, int rows, int& turn) {
    __shared__ int list[kRestList], rank_of_at;
    __shared__ int of_warp[2][8];         // how many positions of this target each warp sees
    __shared__ float4 shared[256];
    const int y = a.pk.target[at], tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (y < 0) return;                // outside the vocabulary: all of dW is NaN already
    const int first = a.pk.first_of[y], most_parts = (a.d + kRestCols - 1) / kRestCols;
    if (first != at && most_parts == 1) return;
    float* sums = a.pk.dw_rows + static_cast<long long>(a.pk.dw_by_position ? first : y) * a.d;
    int seen = 0, count = 0;              // positions of this target, and those listed
    for (int base = first & ~3; base < rows; base += kRestScan, turn ^= 1) {
        if (base <= at && seen >= most_parts) return;         // no part is left for `at`
        const int i = base + tid * 8;
        uint32_t hits = 0;
#pragma unroll
        for (int q = 0; q < 8; q += 4)
            if (i + q < rows) {           // the array goes on to a multiple of 256
                const int4 t = *reinterpret_cast<const int4*>(a.pk.target + i + q);
                hits |= (static_cast<uint32_t>(t.x == y) | static_cast<uint32_t>(t.y == y) << 1 |
                         static_cast<uint32_t>(t.z == y) << 2 | static_cast<uint32_t>(t.w == y) << 3) << q;
            }
        if (i + 8 > rows) hits &= (1u << max(rows - i, 0)) - 1u;
        // this thread's hits come behind those of the threads before it
        int before = 0, all = 0;
        if (__any_sync(0xffffffffu, hits != 0)) {
            before = __popc(hits);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += o;
            }
            all = __shfl_sync(0xffffffffu, before, 31);
            before -= __popc(hits);
        }
        if (lane == 0) of_warp[turn][warp] = all;
        __syncthreads();
        if (base > at && rank_of_at >= most_parts) {
            turn ^= 1;
            return;
        }
        all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const int o = of_warp[turn][w];
            if (w < warp) before += o;
            all += o;
        }
        if (count + all > kRestList) {        // `at` has its part: there are more positions than parts
            add_rest<false>(a, sums, y, list, count, true, rank_of_at, shared);
            __syncthreads();
            count = 0;
        }
        for (; hits; hits &= hits - 1) {
            const int k = i + __ffs(hits) - 1;
            if (k == at) rank_of_at = seen + before;
            list[count + before++] = k;
        }
        seen += all;
        count += all;
    }
    __syncthreads();
    const bool many = seen >= 8;
    const int parts = many ? most_parts : (a.d + 1023) / 1024;
    for (int part = rank_of_at; part < parts; part += seen)
        add_rest<true>(a, sums, y, list, count, many, part, shared);
}

// dh rows: the slabs' sum and the target's remainder in bf16 at the original positions; the rows of dW that are a
// target's (see kRestList).  After a wait that ran out both gradients are NaN.
__global__ void __launch_bounds__(256) dg_xent_finish_kernel(const __grid_constant__ FinishArgs a) {
    griddep_wait();
    griddep_launch();         // not before: the next kernel's CTAs beside these cost 2.7 of 47 us at 256 x 4096 x 128
    const bool bad = *a.pk.err != 0;
    const int rows = *a.pk.count, d = a.d;
    if (bad && a.dw) {
        uint32_t* words = static_cast<uint32_t*>(a.dw);
        const long long step = static_cast<long long>(gridDim.x) * 256;
        for (long long k = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; k < a.dw_words; k += step)
            words[k] = 0x7FFF7FFFu;           // NaN as bf16 and as fp32
    }
    if (static_cast<int>(blockIdx.x) >= a.dh_ctas) {
        const int ctas = static_cast<int>(gridDim.x) - a.dh_ctas;
        int turn = 0;
        for (int at = static_cast<int>(blockIdx.x) - a.dh_ctas; at < rows && !bad; at += ctas)
            finish_dw_row(a, at, rows, turn);
        return;
    }
    const int vecs = d / 4;
    const long long step = static_cast<long long>(a.dh_ctas) * 256;
    for (long long k = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
         k < static_cast<long long>(rows) * vecs; k += step) {
        const int i = static_cast<int>(k / vecs), c = static_cast<int>(k % vecs) * 4;
        const float* src = a.slab + static_cast<long long>(i) * d + c;
        const int y = a.pk.target[i];
        const float t = a.pk.trest[i];
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.W + static_cast<long long>(max(y, 0)) * d + c));
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
        for (int s = 0; s < a.splits; ++s) {
            const float4 u = __ldg(reinterpret_cast<const float4*>(src + s * a.slab_stride));
            x[0] += u.x;
            x[1] += u.y;
            x[2] += u.z;
            x[3] += u.w;
        }
        if (y >= 0) {            // outside the vocabulary: NaN already
            x[0] = fmaf(t, __uint_as_float(w.x << 16), x[0]);
            x[1] = fmaf(t, __uint_as_float(w.x & 0xFFFF0000u), x[1]);
            x[2] = fmaf(t, __uint_as_float(w.y << 16), x[2]);
            x[3] = fmaf(t, __uint_as_float(w.y & 0xFFFF0000u), x[3]);
        }
        uint2 o = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
        if (bad) o = make_uint2(0x7FFF7FFFu, 0x7FFF7FFFu);
        *reinterpret_cast<uint2*>(a.dh + static_cast<long long>(a.pk.row[i]) * d + c) = o;
    }
}

// ------------------------------------------------------------------ host side
struct XentPlan {
    int rows_alloc, v_tiles, d_tiles, pairs;
    int piece, pieces;       // columns per piece of the backward, and their number
    int splits, kb_per_split;
    int dw_by_position;
    size_t err, row, target, lse2, coef, tcoef, trest, first_of, dw_rows, zt2, h, tickets, part, g, slab, total;
};

constexpr int kMaxRows = 1 << 22;
constexpr long long kScratchBytes = 400LL << 20;     // of G in the backward, where the caller names no other

dg_status plan_xent(const dg_xent_params* p, bool backward, XentPlan* out) {
    if (!p || p->n < 0 || p->vocab < 1 || p->hidden < 1) return DG_EINVAL;
    // 1 / T in fp32 too: below 4e-39 it is infinite, and every difference of logits with it
    if (!(p->temperature > 0.f) || !std::isfinite(p->temperature) || !std::isfinite(kLog2e / p->temperature))
        return DG_EINVAL;
    if (p->target_type != DG_INT32 && p->target_type != DG_INT64) return DG_EINVAL;
    if (p->dw_type != DG_BF16 && p->dw_type != DG_FP32) return DG_EINVAL;
    if (p->dw_accumulate != 0 && p->dw_accumulate != 1) return DG_EINVAL;
    if (p->h_stride != 0 && p->h_stride < p->hidden) return DG_EINVAL;
    if (p->scratch_bytes < 0) return DG_EINVAL;
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
    q.trest = take(4 * n);
    q.zt2 = take(4 * n);
    q.h = take(2 * n * p->hidden);
    if (!backward) {
        q.tickets = take(4);
        // (maximum, sum) of every half tile, or of every epilogue warp of the kernel for few positions
        const size_t of_few = p->n <= kFewRows ? sizeof(float2) * 8 * q.pairs * kFewRows : 0;
        q.part = take(16 * n * q.v_tiles > of_few ? 16 * n * q.v_tiles : of_few);
    } else {
        // The whole vocabulary in one piece where G fits the scratch, else pieces whose two buffers do (fewer and
        // longer launches: a training step of 256 positions, V = 262144, d = 2816 took 2.3 ms in pieces of 8704
        // columns, 1.9 ms in pieces of 70000; of 4096 positions 22.5 ms in pieces of 5888, 21.5 ms of 25600).
        const long long scratch = p->scratch_bytes > 0 ? p->scratch_bytes : kScratchBytes;
        const long long column = 2 * static_cast<long long>(q.rows_alloc > 0 ? q.rows_alloc : 1);
        const long long all = static_cast<long long>(q.v_tiles) * kTile;
        long long piece = scratch / (2 * column) / kTile * kTile;
        if (piece < kTile) piece = kTile;
        if (all <= piece || all <= scratch / column) piece = all;
        q.piece = static_cast<int>(piece);
        q.pieces = (p->vocab + q.piece - 1) / q.piece;
        // dh: about one item (two tiles) for every pair, split along the vocabulary into no less than 8 stages
        const int kbs = q.piece / kK;
        const int items = m_tiles * ((q.d_tiles + 1) / 2);
        int splits = items > 0 ? q.pairs / items : 1;
        if (splits > kbs / 8) splits = kbs / 8;
        if (splits < 1) splits = 1;
        q.kb_per_split = (kbs + splits - 1) / splits;
        q.splits = (kbs + q.kb_per_split - 1) / q.kb_per_split;
        q.tickets = take(4 * static_cast<size_t>(q.pieces + 1));
        q.g = take((q.pieces > 1 ? 4 : 2) * n * q.piece);
        q.slab = take(4 * n * p->hidden * q.splits);
        q.first_of = take(4 * static_cast<size_t>(p->vocab));
        q.dw_by_position = p->n < p->vocab;
        q.dw_rows = take(4 * static_cast<size_t>(q.dw_by_position ? p->n : p->vocab) * p->hidden);
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
    k.zt2 = at<float>(ws, q.zt2);
    k.tickets = at<uint32_t>(ws, q.tickets);
    k.n_tickets = q.pieces + 1;
    k.lse2 = at<float>(ws, q.lse2);
    k.coef = at<float>(ws, q.coef);
    k.tcoef = at<float>(ws, q.tcoef);
    k.trest = at<float>(ws, q.trest);
    k.first_of = at<int32_t>(ws, q.first_of);
    k.dw_rows = at<float>(ws, q.dw_rows);
    k.dw_by_position = q.dw_by_position;
    k.h = at<__nv_bfloat16>(ws, q.h);
    return k;
}

// A row-major bf16 matrix with boxes of 64 columns x box_rows rows in 128-byte swizzled rows.
bool encode_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    host::EncodeTiledFn enc = host::encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
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
    if (cudaFuncSetAttribute(dg_xent_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmemBytes) != cudaSuccess)
        return false;
    for (auto k : {dg_xent_gemm_kernel<true>, dg_xent_gemm_kernel<false>})
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) return false;
    done[dev] = true;
    return true;
}

// A kernel that waits (griddepcontrol.wait) for the one before it on the stream: set up while that one runs.
template <class... KArgs, class... Args>
cudaError_t launch_next(void (*kern)(KArgs...), int grid, int block, int cluster, size_t smem, cudaStream_t s,
                        Args&&... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
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

template <bool kForward>
cudaError_t launch_gemm(const GemmArgs& a, long long most_items, int pairs, cudaStream_t s) {
    const int grid = 2 * static_cast<int>(most_items < pairs ? most_items : pairs);
    return launch_next(dg_xent_gemm_kernel<kForward>, grid, kXThreads, 2, kSmemBytes, s, a);
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Ranges [a, a + na) and [b, b + nb) overlap.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

dg_status launch_pack(const PackArgs& in, cudaStream_t s) {
    const int rows = (in.n + kK - 1) / kK * kK;
    PackArgs a = in;
    a.row_ctas = (rows + in.rows_per_cta - 1) / in.rows_per_cta;
    // 16 KB a CTA, on as many as there are pairs at most
    const int clearing = in.clears ? (in.vocab + 4095) / 4096 : 0;
    const int grid = a.row_ctas + (clearing < in.clears ? clearing : in.clears);
    return launch_next(dg_xent_pack_kernel, grid, 256, 1, 0, s, a) == cudaSuccess ? DG_OK : DG_ECUDA;
}

PackArgs pack_args(const dg_xent_params* p, const XentPlan& q, void* ws, const void* h, const void* W,
                   const void* targets) {
    PackArgs a;
    std::memset(&a, 0, sizeof(a));
    a.out = packed_of(q, ws);
    a.h = static_cast<const __nv_bfloat16*>(h);
    a.W = static_cast<const __nv_bfloat16*>(W);
    a.h_stride = p->h_stride ? p->h_stride : p->hidden;
    a.targets = targets;
    a.targets64 = p->target_type == DG_INT64;
    a.ignore = p->ignore_index;
    a.n = p->n;
    a.d = p->hidden;
    a.vocab = p->vocab;
    a.rows_per_cta = kPackRows * ((p->n + 2048 * kPackRows - 1) / (2048 * kPackRows));
    a.inv_t = static_cast<float>(1.0 / static_cast<double>(p->temperature));
    a.scale_log2 = static_cast<float>(1.4426950408889634 / static_cast<double>(p->temperature));
    return a;
}

GemmArgs gemm_args(const dg_xent_params* p, const XentPlan& q, void* ws) {
    GemmArgs a;
    std::memset(&a, 0, sizeof(a));
    a.pk = packed_of(q, ws);
    a.wait_ns = host::counter_wait_ns();
    a.vocab = p->vocab;
    a.d = p->hidden;
    a.d_tiles = q.d_tiles;
    a.wide = 2 * q.pairs;
    a.tail = q.pairs;
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

    PackArgs pa = pack_args(p, q, workspace_dev, h_dev, W_dev, targets_dev);
    pa.loss_out = loss_dev;
    pa.lse_out = lse_dev;
    const Packed pk = pa.out;
    float2* part = at<float2>(workspace_dev, q.part);
    GemmArgs ga;
    FewArgs fa;
    int parts, grid = 0;
    const bool few = p->n <= kFewRows;
    if (few) {
        std::memset(&fa, 0, sizeof(fa));
        fa.pk = pk;
        fa.wait_ns = host::counter_wait_ns();
        fa.vocab = p->vocab;
        fa.d = p->hidden;
        fa.columns = p->n <= 16 ? 16 : kFewRows;
        fa.scale_log2 = pa.scale_log2;
        fa.part = part;
        grid = 2 * static_cast<int>(q.v_tiles < q.pairs ? q.v_tiles : q.pairs);
        parts = 4 * grid;
        if (!encode_2d(&fa.h, pk.h, p->n, p->hidden, fa.columns) || !encode_2d(&fa.w, W_dev, p->vocab, p->hidden, kHalf))
            return DG_ECUDA;
    } else {
        ga = gemm_args(p, q, workspace_dev);
        ga.ticket = pk.tickets;
        ga.tiles_logits = q.v_tiles;
        ga.part = part;
        parts = 2 * q.v_tiles;
        if (!encode_2d(&ga.h_k, pk.h, p->n, p->hidden, kHalf) || !encode_2d(&ga.w_k, W_dev, p->vocab, p->hidden, kHalf))
            return DG_ECUDA;
    }
    const dg_status sp = launch_pack(pa, s);
    if (sp != DG_OK) return sp;
    const long long tiles = static_cast<long long>(q.rows_alloc / kTile) * q.v_tiles;
    const cudaError_t e = few ? launch_next(dg_xent_few_kernel, grid, kFewThreads, 2, kFewSmemBytes, s, fa)
                              : launch_gemm<true>(ga, tiles, q.pairs, s);
    if (e != cudaSuccess) return DG_ECUDA;
    if (launch_next(dg_xent_merge_kernel, p->n, 256, 1, 0, s, pk, static_cast<const float2*>(part), parts, loss_dev,
                    lse_dev) != cudaSuccess)
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
    // the products read W after the first of its gradient's rows are written, and no positions still zero dW
    const size_t w_bytes = static_cast<size_t>(p->vocab) * p->hidden * 2;
    if (dW_dev && W_dev && overlap(dW_dev, dw_bytes, W_dev, w_bytes)) return DG_EINVAL;
    if (p->n == 0) {
        if (dW_dev && !p->dw_accumulate && cudaMemsetAsync(dW_dev, 0, dw_bytes, s) != cudaSuccess) return DG_ECUDA;
        return DG_OK;
    }
    if (!h_dev || !W_dev || !targets_dev || !loss_dev || !lse_dev || !dloss_dev || !workspace_dev) return DG_EINVAL;
    if (!aligned(h_dev, 2) || !aligned(W_dev, 16) || !aligned(targets_dev, p->target_type == DG_INT64 ? 8 : 4) ||
        !aligned(loss_dev, 4) || !aligned(lse_dev, 4) || !aligned(dloss_dev, 4) || !aligned(workspace_dev, 256))
        return DG_EINVAL;
    const size_t dh_bytes = static_cast<size_t>(p->n) * p->hidden * 2;
    const size_t h_bytes = 2 * (static_cast<size_t>(p->n - 1) * (p->h_stride ? p->h_stride : p->hidden) + p->hidden);
    if (dh_dev && (overlap(dh_dev, dh_bytes, W_dev, w_bytes) || overlap(dh_dev, dh_bytes, h_dev, h_bytes)))
        return DG_EINVAL;
    if (dh_dev && dW_dev && overlap(dh_dev, dh_bytes, dW_dev, dw_bytes)) return DG_EINVAL;
    if (workspace_bytes < q.total) return DG_ENOMEM;
    if (!gemm_attr_set()) return DG_ECUDA;

    PackArgs pa = pack_args(p, q, workspace_dev, h_dev, W_dev, targets_dev);
    pa.loss_in = loss_dev;
    pa.lse_in = lse_dev;
    pa.dloss = dloss_dev;
    pa.dh = static_cast<__nv_bfloat16*>(dh_dev);
    pa.clears = dW_dev ? q.pairs : 0;
    GemmArgs ga = gemm_args(p, q, workspace_dev);
    void* g = at<void>(workspace_dev, q.g);
    float* slab = at<float>(workspace_dev, q.slab);
    ga.g_rows = ga.slab_rows = q.rows_alloc;
    ga.kb_per_split = q.kb_per_split;
    ga.want_dh = dh_dev != nullptr;
    ga.want_dw = dW_dev != nullptr;
    ga.slab = slab;
    ga.dw = dW_dev;
    ga.dw_fp32 = p->dw_type == DG_FP32;
    ga.dw_accumulate = p->dw_accumulate;
    const uint64_t rows = q.rows_alloc, d = p->hidden, g_rows = q.pieces > 1 ? 2 * rows : rows;
    if (!encode_2d(&ga.h_k, ga.pk.h, p->n, d, kHalf) || !encode_2d(&ga.h_mn, ga.pk.h, rows, d, kK) ||
        !encode_2d(&ga.w_k, W_dev, p->vocab, d, kHalf) || !encode_2d(&ga.w_mn, W_dev, p->vocab, d, kK) ||
        !encode_2d(&ga.g_k, g, g_rows, q.piece, kHalf) || !encode_2d(&ga.g_mn, g, g_rows, q.piece, kK) ||
        !encode_2d(&ga.g_out, g, g_rows, q.piece, 32) ||
        (dW_dev && !ga.dw_fp32 && !encode_2d(&ga.dw_out, dW_dev, p->vocab, d, 32)))
        return DG_ECUDA;
    // the kinds of tiles, longest contraction first
    const int length[3] = {(p->hidden + kK - 1) / kK, q.kb_per_split, (p->n + kK - 1) / kK};
    const int kind[3] = {kLogits, kDh, kDw};
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (length[order[j]] < length[order[j + 1]]) std::swap(order[j], order[j + 1]);
    for (int i = 0; i < 3; ++i) ga.order[i] = kind[order[i]];

    const dg_status sp = launch_pack(pa, s);
    if (sp != DG_OK) return sp;
    const int m_tiles = q.rows_alloc / kTile;
    auto tiles_of = [&](int piece) {
        const int left = p->vocab - piece * q.piece;
        return ((left < q.piece ? left : q.piece) + kTile - 1) / kTile;
    };
    for (int k = -1; k < q.pieces; ++k) {
        ga.ticket = ga.pk.tickets + (k + 1);
        ga.v0_logits = (k + 1) * q.piece;
        ga.tiles_logits = k + 1 < q.pieces ? tiles_of(k + 1) : 0;
        ga.v0_grads = k * q.piece;
        ga.tiles_grads = k >= 0 ? tiles_of(k) : 0;
        ga.g_write = (k + 1) & 1;
        ga.g_read = k & 1;
        ga.first_piece = k == 0;
        ga.mark = k < 0 && dW_dev;
        // a short last piece may need fewer splits; the slabs left out keep their sums
        ga.splits = (ga.tiles_grads * (kTile / kK) + q.kb_per_split - 1) / q.kb_per_split;
        const long long tiles = static_cast<long long>(m_tiles) * ga.tiles_logits +
                                (ga.want_dh ? static_cast<long long>(m_tiles) * q.d_tiles * ga.splits : 0) +
                                (ga.want_dw ? static_cast<long long>(ga.tiles_grads) * q.d_tiles : 0);
        if (launch_gemm<false>(ga, tiles, q.pairs, s) != cudaSuccess) return DG_ECUDA;
    }
    FinishArgs fa;
    std::memset(&fa, 0, sizeof(fa));
    fa.pk = ga.pk;
    fa.slab = slab;
    fa.slab_stride = static_cast<long long>(rows * d);
    fa.splits = q.splits;
    fa.d = p->hidden;
    fa.W = static_cast<const __nv_bfloat16*>(W_dev);
    fa.dh = static_cast<__nv_bfloat16*>(dh_dev);
    fa.dw = dW_dev;
    fa.dw_words = static_cast<long long>(dw_bytes / 4);
    fa.dw_fp32 = ga.dw_fp32;
    fa.dw_accumulate = p->dw_accumulate;
    // both gradients side by side, 8 CTAs an SM each at most: dh a thread for 4 columns, dW a CTA for a position
    const long long most = q.pairs * 16LL, dh_work = (static_cast<long long>(p->n) * (p->hidden / 4) + 255) / 256;
    fa.dh_ctas = dh_dev ? static_cast<int>(dh_work < most ? dh_work : most) : 0;
    const int dw_ctas = dW_dev ? static_cast<int>(p->n < most ? p->n : most) : 0;
    if (launch_next(dg_xent_finish_kernel, fa.dh_ctas + dw_ctas, 256, 1, 0, s, fa) != cudaSuccess) return DG_ECUDA;
    const int launches = q.pieces + 2;
    set_last_launches(launches + 1);
    return DG_OK;
}

}  // extern "C"
