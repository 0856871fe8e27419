// AdamW with decoupled weight decay over many tensors in one launch, with first and second moments
// in fp32 or in 8 bits.
//
// Per element, with g' = grad_scale g and step t:
//   m <- b1 m + (1 - b1) g'      v <- b2 v + (1 - b2) g'^2
//   p <- p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// all in fp32; the update uses the new moments before they are stored.
//
// 8-bit states: m and r = sqrt(v) of every 256 consecutive elements are E4M3 codes times one power
// of two 2^e (e the smallest with max |x| 2^-e <= 448, as dg_quantize_e4m3 picks it; 0 for a block
// of zeros, at least -100).  The root is stored because its range is half of v's in octaves.  Codes
// are rounded at random between the two E4M3 neighbours, up with the probability of the distance
// from the lower one: a code's half step is 2^-4 of the value, far more than the (1 - b2) by which
// one step moves v, so rounding to nearest would never let a state drift.  A positive root is stored
// as at least the smallest code (a zero there would divide m by eps).  Non-finite values are stored
// as NaN.  bf16 parameters without an fp32 master can be rounded the same way, for the same reason.
//
// Bound: bytes (the bf16 parameter with 8-bit states moves 10 bytes an element, the fp32 one with
// fp32 states 28).  One warp owns one 256-element block, 8 consecutive elements a lane, so the
// block's maxima are a 5-step shuffle and every access is 8 (codes), 16 (bf16) or 32 bytes (fp32) a
// lane.  The list of tensors travels in the kernel's argument (no copy, nothing to keep alive until
// the launch has run, and a captured graph holds its own list); a CTA finds its tensor by bisection.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/dg.h"
#include "dg_common.cuh"
#include "dg_host.h"

namespace dg {

namespace {

constexpr int kBlock = 256;           // elements that share an exponent: one warp, 8 a lane
constexpr int kWarps = 8;
constexpr int kMinExp = -100;         // 2^-e and 2^(e - 9) stay normal
constexpr uint32_t kTagState = 5, kTagParam = 6;
constexpr int kFewTensors = 24;       // the short list's argument is under 2 KB
constexpr int kManyTensors = 400;     // the long one's under the 32764 bytes a launch can pass

struct Tensor {
    void* param;
    const void* grad;
    void* m;
    void* v;
    int8_t* m_exp;
    int8_t* v_exp;
    float* master;
    long long n;
    float weight_decay;
    int aligned;                      // every pointer allows the 8-element accesses
};

template <int kCap>
struct Args {
    double lr, beta1, beta2;
    float b1, one_minus_b1, b2, one_minus_b2, eps;
    float step_size, inv_root_bc2;    // lr / (1 - b1^t), 1 / sqrt(1 - b2^t); with step_dev computed on the device
    float grad_scale;
    const float* lr_dev;
    const int32_t* step_dev;
    const float* grad_scale_dev;
    uint32_t seed_lo, seed_hi, step, first_tensor;
    int stochastic, n_tensors, blocks_per_warp;
    Tensor t[kCap];
    int first_cta[kCap + 1];
};

// 8 elements of a lane as fp32 <-> memory, `live` of them in range (8 with vectors only).
__device__ __forceinline__ void load8(const float* p, bool vec, int live, float (&x)[8]) {
    if (vec) {
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < live ? p[i] : 0.f;
    }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, bool vec, int live, float (&x)[8]) {
    if (vec) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < live ? __bfloat162float(p[i]) : 0.f;
    }
}

__device__ __forceinline__ void store8(float* p, bool vec, int live, const float (&x)[8]) {
    if (vec) {
        asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                     "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "l"(p)
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = x[i];
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, bool vec, int live, const float (&x)[8]) {
    if (vec) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// 8 codes of a lane as two words.
__device__ __forceinline__ void load_codes(const uint8_t* p, bool vec, int live, uint32_t (&c)[2]) {
    if (vec) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        c[0] = w.x;
        c[1] = w.y;
    } else {
        c[0] = c[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) c[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
    }
}

__device__ __forceinline__ void store_codes(uint8_t* p, bool vec, int live, const uint32_t (&c)[2]) {
    if (vec) {
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
    }
}

// x = E4M3 codes times 2^e (exact: e >= -100 keeps every product normal).
__device__ __forceinline__ void decode8(const uint32_t (&c)[2], int e, float (&x)[8]) {
    const float scale = __int_as_float((e + 127) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t pair = static_cast<__nv_fp8x2_storage_t>(c[i >> 1] >> (16 * (i & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[2 * i] = f.x * scale;
        x[2 * i + 1] = f.y * scale;
    }
}

// The exponent of a block whose lane maxima of |x| (finite ones only) are `peak`: the smallest e
// with max 2^-e <= 448 = 1.75 2^8 (a significand above 1.75 takes the next exponent).
__device__ __forceinline__ int block_exponent(float peak) {
    const int bits = __reduce_max_sync(0xffffffffu, __float_as_int(peak));
    if (bits == 0) return 0;
    const int e = ((bits + 0x1FFFFF) >> 23) - 135;
    return e < kMinExp ? kMinExp : e;
}

// |x| 2^-e as an E4M3 code, rounded up when the discarded part and the 16 random bits u carry.
// Below the smallest normal 2^-6 the sum with 2^-6 has the subnormals' spacing.
__device__ __forceinline__ uint32_t round_e4m3(float ax, float inv_scale, uint32_t u) {
    if (!(ax < INFINITY)) return 0x7Fu;
    const float y = ax * inv_scale;
    const bool small = y < 0.015625f;
    const uint32_t b = __float_as_uint(small ? y + 0.015625f : y) + (u << 4);
    return (b >> 20) - (small ? 968u : 960u);
}

__device__ __forceinline__ float finite_max(float peak, float ax) { return ax < INFINITY ? fmaxf(peak, ax) : peak; }

template <class P, class G, bool kState8, bool kMaster, int kCap>
__global__ void __launch_bounds__(kWarps * 32) dg_adamw_kernel(const __grid_constant__ Args<kCap> a) {
    // the tensor this CTA works on
    int lo = 0, hi = a.n_tensors;
    const int cta = blockIdx.x;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first_cta[mid] <= cta) lo = mid;
        else hi = mid;
    }
    const Tensor& t = a.t[lo];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    double lr = a.lr;
    float step_size = a.step_size, inv_root_bc2 = a.inv_root_bc2, gscale = a.grad_scale;
    uint32_t step = a.step;
    if (a.grad_scale_dev) gscale *= *a.grad_scale_dev;
    if (a.lr_dev) lr = static_cast<double>(*a.lr_dev);
    if (a.step_dev || a.lr_dev) {
        __shared__ double corr[2];
        if (a.step_dev) step = static_cast<uint32_t>(*a.step_dev);
        if (threadIdx.x == 0) {
            // 1 - b^t without cancellation; b = 0 gives 1
            corr[0] = a.beta1 > 0 ? -expm1(step * log(a.beta1)) : 1.0;
            corr[1] = a.beta2 > 0 ? -expm1(step * log(a.beta2)) : 1.0;
        }
        __syncthreads();
        step_size = static_cast<float>(lr / corr[0]);
        inv_root_bc2 = static_cast<float>(1.0 / sqrt(corr[1]));
    }
    const float keep = static_cast<float>(1.0 - lr * static_cast<double>(t.weight_decay));

    const long long n = t.n;
    const long long first = static_cast<long long>(cta - a.first_cta[lo]) * a.blocks_per_warp * kWarps;
    for (int k = 0; k < a.blocks_per_warp; ++k) {
        // neighbouring warps on neighbouring blocks, so that a CTA's accesses are one run of memory
        const long long blk = first + static_cast<long long>(k) * kWarps + warp;
        const long long at = blk * kBlock + lane * 8;
        if (blk * kBlock >= n) break;
        const int live = at >= n ? 0 : (n - at < 8 ? static_cast<int>(n - at) : 8);
        const bool vec = t.aligned && live == 8;

        float p[8], g[8], m[8], v[8];
        if constexpr (kMaster) load8(t.master + at, vec, live, p);
        else load8(static_cast<const P*>(t.param) + at, vec, live, p);
        load8(static_cast<const G*>(t.grad) + at, vec, live, g);
        if constexpr (kState8) {
            uint32_t cm[2], cv[2];
            load_codes(static_cast<const uint8_t*>(t.m) + at, vec, live, cm);
            load_codes(static_cast<const uint8_t*>(t.v) + at, vec, live, cv);
            decode8(cm, t.m_exp[blk], m);
            decode8(cv, t.v_exp[blk], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
        } else {
            load8(static_cast<const float*>(t.m) + at, vec, live, m);
            load8(static_cast<const float*>(t.v) + at, vec, live, v);
        }

        // moments with every product and sum rounded by itself, so that the stored states do not
        // depend on how the compiler contracts them
        float peak_m = 0.f, peak_r = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gi = __fmul_rn(g[i], gscale);
            m[i] = __fadd_rn(__fmul_rn(m[i], a.b1), __fmul_rn(gi, a.one_minus_b1));
            v[i] = __fadd_rn(__fmul_rn(v[i], a.b2), __fmul_rn(__fmul_rn(gi, gi), a.one_minus_b2));
            const float r = __fsqrt_rn(v[i]);
            p[i] = fmaf(p[i], keep, -__fdividef(m[i] * step_size, fmaf(r, inv_root_bc2, a.eps)));
            if constexpr (kState8) {
                v[i] = r;
                peak_m = finite_max(peak_m, fabsf(m[i]));
                peak_r = finite_max(peak_r, r);
            }
        }

        if constexpr (kMaster) {
            store8(t.master + at, vec, live, p);
            store8(static_cast<P*>(t.param) + at, vec, live, p);
        } else {
            if constexpr (sizeof(P) == 2) {
                if (a.stochastic) {
                    uint32_t w[4] = {static_cast<uint32_t>(at >> 3), step, a.first_tensor + lo, kTagParam};
                    philox4x32_10(w, a.seed_lo, a.seed_hi);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t u = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
                        if (fabsf(p[i]) < INFINITY)
                            p[i] = __uint_as_float((__float_as_uint(p[i]) + u) & 0xFFFF0000u);
                    }
                }
            }
            store8(static_cast<P*>(t.param) + at, vec, live, p);
        }
        if constexpr (kState8) {
            const int em = block_exponent(peak_m), er = block_exponent(peak_r);
            const float sm = __int_as_float((127 - em) << 23), sr = __int_as_float((127 - er) << 23);
            uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t w[4] = {static_cast<uint32_t>((at >> 2) + q), step, a.first_tensor + lo, kTagState};
                philox4x32_10(w, a.seed_lo, a.seed_hi);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float mi = m[4 * q + i], ri = v[4 * q + i];
                    const uint32_t sign = (__float_as_uint(mi) >> 31 && mi != 0.f) ? 0x80u : 0u;
                    cm[q] |= (round_e4m3(fabsf(mi), sm, w[i] & 0xFFFFu) | sign) << (8 * i);
                    const uint32_t c = round_e4m3(ri, sr, w[i] >> 16);
                    cv[q] |= (c == 0u && ri > 0.f ? 1u : c) << (8 * i);
                }
            }
            store_codes(static_cast<uint8_t*>(t.m) + at, vec, live, cm);
            store_codes(static_cast<uint8_t*>(t.v) + at, vec, live, cv);
            if (lane == 0) {
                t.m_exp[blk] = static_cast<int8_t>(em);
                t.v_exp[blk] = static_cast<int8_t>(er);
            }
        } else {
            store8(static_cast<float*>(t.m) + at, vec, live, m);
            store8(static_cast<float*>(t.v) + at, vec, live, v);
        }
    }
}

template <class P, class G, bool kState8, bool kMaster, int kCap>
cudaError_t launch(const Args<kCap>& a, int n_ctas, cudaStream_t s) {
    dg_adamw_kernel<P, G, kState8, kMaster, kCap><<<n_ctas, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <class P, class G, int kCap>
cudaError_t launch_types(const Args<kCap>& a, bool state8, bool master, int n_ctas, cudaStream_t s) {
    if constexpr (sizeof(P) == 2) {
        if (master)
            return state8 ? launch<P, G, true, true>(a, n_ctas, s) : launch<P, G, false, true>(a, n_ctas, s);
    }
    return state8 ? launch<P, G, true, false>(a, n_ctas, s) : launch<P, G, false, false>(a, n_ctas, s);
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Launch the tensors [begin, end) as one grid; returns the status.
template <int kCap>
dg_status launch_range(const dg_adamw_params* p, const dg_adamw_tensor* tensors, int begin, int end,
                       int blocks_per_warp, cudaStream_t s) {
    Args<kCap> a;
    std::memset(&a, 0, sizeof(a));
    a.lr = p->lr;
    a.beta1 = p->beta1;
    a.beta2 = p->beta2;
    a.b1 = static_cast<float>(p->beta1);
    a.one_minus_b1 = static_cast<float>(1.0 - p->beta1);
    a.b2 = static_cast<float>(p->beta2);
    a.one_minus_b2 = static_cast<float>(1.0 - p->beta2);
    a.eps = static_cast<float>(p->eps);
    if (!p->step_dev) {
        a.step_size = static_cast<float>(p->lr / (1.0 - std::pow(p->beta1, p->step)));
        a.inv_root_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(p->beta2, p->step)));
    }
    a.grad_scale = p->grad_scale;
    a.lr_dev = p->lr_dev;
    a.step_dev = p->step_dev;
    a.grad_scale_dev = p->grad_scale_dev;
    a.seed_lo = static_cast<uint32_t>(p->seed);
    a.seed_hi = static_cast<uint32_t>(p->seed >> 32);
    a.step = static_cast<uint32_t>(p->step);
    a.first_tensor = static_cast<uint32_t>(begin);
    a.stochastic = p->stochastic;
    a.blocks_per_warp = blocks_per_warp;
    a.n_tensors = end - begin;
    const long long per_cta = static_cast<long long>(kBlock) * kWarps * blocks_per_warp;
    long long ctas = 0;
    const uintptr_t pa = p->param_type == DG_FP32 ? 32 : 16, ga = p->grad_type == DG_FP32 ? 32 : 16;
    const uintptr_t sa = p->state_bits == 8 ? 8 : 32;
    bool master = false;
    for (int i = begin; i < end; ++i) {
        const dg_adamw_tensor& x = tensors[i];
        Tensor& t = a.t[i - begin];
        t.param = x.param;
        t.grad = x.grad;
        t.m = x.m;
        t.v = x.v;
        t.m_exp = x.m_exp;
        t.v_exp = x.v_exp;
        t.master = x.master;
        t.n = x.n;
        t.weight_decay = x.weight_decay;
        t.aligned = !(misaligned(x.param, pa) || misaligned(x.grad, ga) || misaligned(x.m, sa) ||
                      misaligned(x.v, sa) || misaligned(x.master, 32));
        master = master || x.master;
        a.first_cta[i - begin] = static_cast<int>(ctas);
        ctas += (x.n + per_cta - 1) / per_cta;       // under 2^31: n < 2^34 and 8192 elements a CTA for long lists
    }
    a.first_cta[end - begin] = static_cast<int>(ctas);
    if (ctas == 0) return DG_OK;
    const int n = static_cast<int>(ctas);
    const bool s8 = p->state_bits == 8;
    cudaError_t e;
    if (p->param_type == DG_FP32)
        e = p->grad_type == DG_FP32 ? launch_types<float, float>(a, s8, false, n, s)
                                    : launch_types<float, __nv_bfloat16>(a, s8, false, n, s);
    else
        e = p->grad_type == DG_FP32 ? launch_types<__nv_bfloat16, float>(a, s8, master, n, s)
                                    : launch_types<__nv_bfloat16, __nv_bfloat16>(a, s8, master, n, s);
    return e == cudaSuccess ? DG_OK : DG_ECUDA;
}

}  // namespace

}  // namespace dg

using namespace dg;
using namespace dg::host;

extern "C" {

void dg_adamw_params_default(dg_adamw_params* p) {
    if (!p) return;
    std::memset(p, 0, sizeof(*p));
    p->lr = 1e-3;
    p->beta1 = 0.9;
    p->beta2 = 0.999;
    p->eps = 1e-8;
    p->grad_scale = 1.0f;
    p->step = 1;
    p->state_bits = 32;
    p->param_type = DG_BF16;
    p->grad_type = DG_BF16;
}

dg_status dg_adamw_step(const dg_adamw_params* p, const dg_adamw_tensor* tensors, int n_tensors, void* stream) {
    set_last_launches(0);
    if (!p || n_tensors < 0 || (n_tensors > 0 && !tensors)) return DG_EINVAL;
    if (!(p->lr >= 0) || !std::isfinite(p->lr) || !(p->beta1 >= 0 && p->beta1 < 1) ||
        !(p->beta2 >= 0 && p->beta2 < 1) || !(p->eps >= 0) || !std::isfinite(p->eps))
        return DG_EINVAL;
    if (!p->step_dev && p->step < 1) return DG_EINVAL;
    if (p->state_bits != 8 && p->state_bits != 32) return DG_EINVAL;
    if ((p->param_type != DG_FP32 && p->param_type != DG_BF16) || (p->grad_type != DG_FP32 && p->grad_type != DG_BF16))
        return DG_EINVAL;
    if (p->stochastic != 0 && (p->stochastic != 1 || p->param_type != DG_BF16)) return DG_EINVAL;
    if (misaligned(p->lr_dev, 4) || misaligned(p->step_dev, 4) || misaligned(p->grad_scale_dev, 4)) return DG_EINVAL;
    const uintptr_t ps = p->param_type == DG_FP32 ? 4 : 2, gs = p->grad_type == DG_FP32 ? 4 : 2;
    const uintptr_t ss = p->state_bits == 8 ? 1 : 4;
    long long total = 0;
    int with_master = 0, live = 0;
    for (int i = 0; i < n_tensors; ++i) {
        const dg_adamw_tensor& x = tensors[i];
        if (x.n < 0 || x.n >= (1LL << 34)) return DG_EINVAL;     // element / 4 is one counter word
        if (!std::isfinite(x.weight_decay)) return DG_EINVAL;
        if (x.n == 0) continue;
        if (!x.param || !x.grad || !x.m || !x.v) return DG_EINVAL;
        if (p->state_bits == 8 && (!x.m_exp || !x.v_exp)) return DG_EINVAL;
        if (misaligned(x.param, ps) || misaligned(x.grad, gs) || misaligned(x.m, ss) || misaligned(x.v, ss) ||
            misaligned(x.master, 4))
            return DG_EINVAL;
        total += x.n;
        ++live;
        with_master += x.master != nullptr;
    }
    // a master copy for all tensors of a call or for none, and only beside bf16 parameters that it rounds to
    if (with_master != 0 && (with_master != live || p->param_type != DG_BF16 || p->stochastic)) return DG_EINVAL;
    // Few elements: one block a warp, to spread them over the SMs.  Many: 4 blocks a warp, which
    // shares a CTA's search of the list over more work.
    const int sms = device_sm_count();
    if (sms <= 0) return DG_ECUDA;
    const int bpw = total > static_cast<long long>(sms) * 8 * kWarps * kBlock * 4 ? 4 : 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    for (int begin = 0; begin < n_tensors;) {
        const int left = n_tensors - begin;
        const int end = begin + (left > kManyTensors ? kManyTensors : left);
        const dg_status st = left <= kFewTensors ? launch_range<kFewTensors>(p, tensors, begin, end, bpw, s)
                                                 : launch_range<kManyTensors>(p, tensors, begin, end, bpw, s);
        if (st != DG_OK) return st;
        ++launches;
        begin = end;
    }
    set_last_launches(launches);
    return DG_OK;
}

}  // extern "C"
