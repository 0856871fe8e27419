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
#include <type_traits>

#include "../../include/dg.h"
#include "dg_common.cuh"
#include "dg_host.h"

namespace dg {

namespace {

constexpr int kBlock = 256;           // elements that share an exponent: one warp, 8 a lane
constexpr int kWarps = 8;
constexpr int kMaxBlocksPerWarp = 8;
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
    float decay;                      // 1 - lr wd; wd itself when lr or the step is on the device
    int aligned;                      // every pointer allows the 8-element accesses
};

// Philox4x32-10 (see dg_common.cuh) with the keys of its rounds made on the host: read from the
// kernel's constants they cost neither registers nor the additions.
struct Keys {
    uint32_t k[10][2];
};

__device__ __forceinline__ void philox(uint32_t (&c)[4], const Keys& keys) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c[0];
        const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
        c[0] = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ keys.k[r][0];
        c[1] = static_cast<uint32_t>(p1);
        c[2] = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ keys.k[r][1];
        c[3] = static_cast<uint32_t>(p0);
    }
}

template <int kCap>
struct Args {
    double lr, beta1, beta2;
    float b1, one_minus_b1, b2, one_minus_b2, eps;
    float step_size, inv_root_bc2;    // lr / (1 - b1^t), 1 / sqrt(1 - b2^t); with step_dev computed on the device
    float grad_scale;
    const float* lr_dev;
    const int32_t* step_dev;
    const float* grad_scale_dev;
    uint32_t step, first_tensor;
    int stochastic, n_tensors, blocks_per_warp;
    Keys keys;
    Tensor t[kCap];
    int first_cta[kCap + 1];
};

// A lane's 8 elements as they lie in memory: 2 (codes), 4 (bf16) or 8 (fp32) words, in one access when
// kVec, else element by element with `live` of them in range (the others 0).
template <class T>
struct Raw8 {
    uint32_t w[2 * sizeof(T)];
};

template <bool kVec, class T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* p, int live) {
    if constexpr (kVec && sizeof(T) == 4) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
                       "=r"(r.w[6]), "=r"(r.w[7])
                     : "l"(p));
    } else if constexpr (kVec && sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
    } else if constexpr (kVec) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        r.w[0] = u.x, r.w[1] = u.y;
    } else {
        constexpr int per = 4 / sizeof(T), bits = 8 * sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / per; ++i) r.w[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) {
                uint32_t x;
                if constexpr (sizeof(T) == 4) x = reinterpret_cast<const uint32_t*>(p)[i];
                else if constexpr (sizeof(T) == 2) x = reinterpret_cast<const uint16_t*>(p)[i];
                else x = reinterpret_cast<const uint8_t*>(p)[i];
                r.w[i / per] |= x << (bits * (i % per));
            }
    }
}

template <bool kVec, class T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r, int live) {
    if constexpr (kVec && sizeof(T) == 4) {
        asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                     "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7]), "l"(p)
                     : "memory");
    } else if constexpr (kVec && sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else if constexpr (kVec) {
        *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    } else {
        constexpr int per = 4 / sizeof(T), bits = 8 * sizeof(T);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) {
                const uint32_t x = r.w[i / per] >> (bits * (i % per));
                if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[i] = x;
                else if constexpr (sizeof(T) == 2) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(x);
                else reinterpret_cast<uint8_t*>(p)[i] = static_cast<uint8_t>(x);
            }
    }
}

__device__ __forceinline__ void to_floats(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
}

__device__ __forceinline__ void to_floats(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r.w[i] << 16);
        x[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void from_floats(Raw8<float>& r, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(x[i]);
}

__device__ __forceinline__ void from_floats(Raw8<__nv_bfloat16>& r, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
}

// Two fp32 values in one register pair: sm_100 multiplies and adds both in one instruction, each
// rounded by itself.
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpack2(f32x2 x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Largest |x|, NaN when one of them is NaN.
__device__ __forceinline__ float peak3(float peak, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(peak), "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float sqrt_sfu(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float div_sfu(float a, float b) {
    float r;
    asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The E4M3 values of a lane's 8 codes.
__device__ __forceinline__ void decode8(const Raw8<uint8_t>& c, f32x2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t pair = static_cast<__nv_fp8x2_storage_t>(c.w[i >> 1] >> (16 * (i & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[i] = pack2(f.x, f.y);
    }
}

// The smallest e with peak 2^-e <= 448 = 1.75 2^8 for the bits of a finite peak >= 0 (a significand
// above 1.75 takes the next exponent).
__device__ __forceinline__ int exponent_of(int bits) {
    if (bits == 0) return 0;
    const int e = ((bits + 0x1FFFFF) >> 23) - 135;
    return e < kMinExp ? kMinExp : e;
}

// The same for sqrt(v), from v's bits: v 4^-e <= 448^2 = 1.53125 2^17.  (No float v above 448^2 4^e has a
// root that rounds to 448 2^e: the next one's root lies more than half a step above it.)
__device__ __forceinline__ int root_exponent_of(int bits) {
    if (bits < 0x00800000) return exponent_of(__float_as_int(__fsqrt_rn(__int_as_float(bits))));
    const int e = (((bits + 0x3BFFFF) >> 23) - 143) >> 1;
    return e < kMinExp ? kMinExp : e;
}

// y in [0, 448] and 16 random bits at [8, 24) of u8 -> the E4M3 code in the top byte's low 7 bits,
// off by 64: 16 (bits of y + 16 u) has the 3 leading significand bits and 4 of the exponent there,
// and the discarded part carries when it and u say so.  Below the smallest normal 2^-6 the
// subnormals' spacing is that of y + 2^-6, whose code is one exponent too high; halving it corrects that.
__device__ __forceinline__ uint32_t e4m3_top(float y, uint32_t u8) {
    if (y < 0.015625f) y = fmaf(y, 0.5f, 0.0078125f);
    return (__float_as_uint(y) << 4) + u8;
}

__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// One value with the checks that e4m3_top leaves out: blocks that hold a NaN or an infinity.
__device__ __noinline__ uint32_t e4m3_careful(float x, int e, uint32_t u8) {
    const float ax = fabsf(x);
    if (!(ax < INFINITY)) return 0x7Fu;
    return ((e4m3_top(ax * pow2(-e), u8) >> 24) & 0x7Fu) ^ 0x40u;
}

// What every element of a tensor's step needs.
struct Step {
    float b1, b2, c1, c2, eps;            // betas, 1 - betas
    float rate, bias, keep, gscale;       // -lr / (1 - b1^t), 1 / sqrt(1 - b2^t), 1 - lr wd
    uint32_t step, tensor;
    int stochastic;
};

// A lane's first element in every array of a tensor.
template <class P, class G, bool kState8>
struct Bases {
    typedef typename std::conditional<kState8, uint8_t, float>::type State;
    P* param;
    const G* grad;
    State *m, *v;
    float* master;
    uint32_t eighth;          // its place / 8
    __device__ __forceinline__ Bases(const Tensor& t, long long at)
        : param(static_cast<P*>(t.param) + at), grad(static_cast<const G*>(t.grad) + at),
          m(static_cast<State*>(t.m) + at), v(static_cast<State*>(t.v) + at), master(t.master + at),
          eighth(static_cast<uint32_t>(at >> 3)) {}
};

// A lane's share of one block: read by load(), written by update(), `at` elements behind its first.
template <class P, class G, bool kState8, bool kMaster>
struct Lane {
    typedef typename std::conditional<kMaster, float, P>::type Source;
    typedef typename std::conditional<kState8, uint8_t, float>::type State;
    Raw8<Source> p;
    Raw8<G> g;
    Raw8<State> m, v;

    template <bool kVec>
    __device__ __forceinline__ void load(const Bases<P, G, kState8>& t, int at, int live) {
        if constexpr (kMaster) load8<kVec>(p, t.master + at, live);
        else load8<kVec>(p, t.param + at, live);
        load8<kVec>(g, t.grad + at, live);
        load8<kVec>(m, t.m + at, live);
        load8<kVec>(v, t.v + at, live);
    }

    template <bool kVec>
    __device__ __forceinline__ void update(const Bases<P, G, kState8>& t, const Step& a, const Keys& keys, int at, int live,
                                           int& em, int& ev) const {
        float px[8], gx[8], mx[8], vx[8], r[8];
        to_floats(p, px);
        to_floats(g, gx);
        f32x2 m2[4], v2[4];          // m and v from before, times b1 and b2
        const f32x2 b1 = pack2(a.b1, a.b1), b2 = pack2(a.b2, a.b2);
        if constexpr (kState8) {
            // a code has 4 significant bits and the scales are powers of two (a value is no less than 2^-109),
            // so that code 2^e is exact, and so is the scale's product with b1
            decode8(m, m2);
            decode8(v, v2);
            const float sm = pow2(em), sv = pow2(ev);
            const f32x2 scaled_b1 = mul2(b1, pack2(sm, sm)), scale_v = pack2(sv, sv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m2[i] = mul2(m2[i], scaled_b1);
                v2[i] = mul2(v2[i], scale_v);
                v2[i] = mul2(mul2(v2[i], v2[i]), b2);
            }
        } else {
            to_floats(m, mx);
            to_floats(v, vx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m2[i] = mul2(pack2(mx[2 * i], mx[2 * i + 1]), b1);
                v2[i] = mul2(pack2(vx[2 * i], vx[2 * i + 1]), b2);
            }
        }
        if (a.gscale != 1.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) gx[i] = __fmul_rn(gx[i], a.gscale);
        }

        // Moments with every product and sum rounded by itself, so that the stored states do not depend on
        // how the compiler contracts them (a product and a sum of two f32x2 may become one fma2: the sums
        // stay scalar).
        const f32x2 rate = pack2(a.rate, a.rate), bias = pack2(a.bias, a.bias), eps = pack2(a.eps, a.eps);
        const f32x2 keep = pack2(a.keep, a.keep), c1 = pack2(a.c1, a.c1), c2 = pack2(a.c2, a.c2);
        float peak_m = 0.f, peak_v = 0.f, peak_p = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 gi = pack2(gx[2 * i], gx[2 * i + 1]);
            float x[2], y[2], u[2], w[2];
            unpack2(m2[i], x[0], x[1]);
            unpack2(mul2(gi, c1), y[0], y[1]);
            unpack2(v2[i], u[0], u[1]);
            unpack2(mul2(mul2(gi, gi), c2), w[0], w[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mx[2 * i + j] = __fadd_rn(x[j], y[j]);
                vx[2 * i + j] = __fadd_rn(u[j], w[j]);
            }
        }
        // The flushing SFU root, which takes a subnormal for 0.  Lanes that hold one (gradients of about 1e-18), or
        // a 0, scale it into the normal range first; the roots themselves are normal.  262144 x 2816 bf16 parameters
        // with 8-bit states: 1.91 ms without this, 1.92 with it, 1.94 with the root that keeps subnormals everywhere.
        float least = vx[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) least = fminf(least, vx[i]);
        if (least < 0x1p-126f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool tiny = vx[i] < 0x1p-126f;
                r[i] = sqrt_sfu(tiny ? vx[i] * 0x1p64f : vx[i]) * (tiny ? 0x1p-32f : 1.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = sqrt_sfu(vx[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[2], y[2];
            unpack2(mul2(pack2(mx[2 * i], mx[2 * i + 1]), rate), x[0], x[1]);
            unpack2(fma2(pack2(r[2 * i], r[2 * i + 1]), bias, eps), y[0], y[1]);
            unpack2(fma2(pack2(px[2 * i], px[2 * i + 1]), keep, pack2(div_sfu(x[0], y[0]), div_sfu(x[1], y[1]))),
                    px[2 * i], px[2 * i + 1]);
            if constexpr (kState8) {
                peak_m = peak3(peak_m, mx[2 * i], mx[2 * i + 1]);
                peak_v = peak3(peak_v, vx[2 * i], vx[2 * i + 1]);
            }
            if constexpr (sizeof(P) == 2 && !kMaster) peak_p = peak3(peak_p, px[2 * i], px[2 * i + 1]);
        }

        Raw8<P> out;
        from_floats(out, px);
        if constexpr (kMaster) {
            Raw8<float> full;
            from_floats(full, px);
            store8<kVec>(t.master + at, full, live);
        } else if constexpr (sizeof(P) == 2) {
            if (a.stochastic) {
                uint32_t w[4] = {t.eighth + at / 8, a.step, a.tensor, kTagParam};
                philox(w, keys);
                if (!(peak_p < INFINITY)) {       // a sum must not carry out of a NaN: no random bits there
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!(fabsf(px[i]) < INFINITY)) w[i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    out.w[i] = __byte_perm(__float_as_uint(px[2 * i]) + (w[i] & 0xFFFFu),
                                           __float_as_uint(px[2 * i + 1]) + (w[i] >> 16), 0x7632);
            }
        }
        store8<kVec>(t.param + at, out, live);

        if constexpr (!kState8) {
            Raw8<float> x;
            from_floats(x, mx);
            store8<kVec>(t.m + at, x, live);
            from_floats(x, vx);
            store8<kVec>(t.v + at, x, live);
        } else {
            int top_m = __reduce_max_sync(0xffffffffu, __float_as_int(peak_m));
            int top_v = __reduce_max_sync(0xffffffffu, __float_as_int(peak_v));
            const bool careful = top_m >= 0x7F800000 || top_v >= 0x7F800000;
            if (careful) {       // the exponents are those of the finite values
                peak_m = peak_v = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (fabsf(mx[i]) < INFINITY) peak_m = fmaxf(peak_m, fabsf(mx[i]));
                    if (vx[i] < INFINITY) peak_v = fmaxf(peak_v, vx[i]);
                }
                top_m = __reduce_max_sync(0xffffffffu, __float_as_int(peak_m));
                top_v = __reduce_max_sync(0xffffffffu, __float_as_int(peak_v));
            }
            // the SFU roots are off by 2^-23 at most, too little to carry a value at the peak over its code
            const int xm = exponent_of(top_m), xr = root_exponent_of(top_v);
            const f32x2 sm = pack2(pow2(-xm), pow2(-xm)), sr = pack2(pow2(-xr), pow2(-xr));
            Raw8<uint8_t> cm, cv;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t w[4] = {2 * (t.eighth + at / 8) + q, a.step, a.tensor, kTagState};
                philox(w, keys);
                uint32_t tm[4], tv[4];
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int j = 4 * q + i;
                    float y[2], z[2];
                    unpack2(mul2(pack2(mx[j], mx[j + 1]), sm), y[0], y[1]);
                    unpack2(mul2(pack2(r[j], r[j + 1]), sr), z[0], z[1]);
                    tm[i] = e4m3_top(fabsf(y[0]), __byte_perm(w[i], 0, 0x4104));
                    tm[i + 1] = e4m3_top(fabsf(y[1]), __byte_perm(w[i + 1], 0, 0x4104));
                    tv[i] = e4m3_top(z[0], __byte_perm(w[i], 0, 0x4324));
                    tv[i + 1] = e4m3_top(z[1], __byte_perm(w[i + 1], 0, 0x4324));
                }
                const uint32_t sign = top_bytes(__float_as_uint(mx[4 * q]), __float_as_uint(mx[4 * q + 1]),
                                                __float_as_uint(mx[4 * q + 2]), __float_as_uint(mx[4 * q + 3]));
                cm.w[q] = ((top_bytes(tm[0], tm[1], tm[2], tm[3]) & 0x7F7F7F7Fu) ^ 0x40404040u) | (sign & 0x80808080u);
                const uint32_t c = (top_bytes(tv[0], tv[1], tv[2], tv[3]) & 0x7F7F7F7Fu) ^ 0x40404040u;
                cv.w[q] = c;
                if ((c - 0x01010101u) & ~c & 0x80808080u) {      // a code of 0: only for a root of 0
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (vx[4 * q + i] > 0.f && (c >> (8 * i) & 0xFFu) == 0) cv.w[q] |= 1u << (8 * i);
                }
                if (careful) {
                    cm.w[q] = sign & 0x80808080u;
                    cv.w[q] = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float vi = vx[4 * q + i];
                        cm.w[q] |= e4m3_careful(mx[4 * q + i], xm, w[i] << 8 & 0xFFFF00u) << (8 * i);
                        const uint32_t k = e4m3_careful(vi < INFINITY ? r[4 * q + i] : NAN, xr, w[i] >> 8 & 0xFFFF00u);
                        cv.w[q] |= (k == 0u && vi > 0.f ? 1u : k) << (8 * i);
                    }
                }
            }
            store8<kVec>(t.m + at, cm, live);
            store8<kVec>(t.v + at, cv, live);
            em = xm;
            ev = xr;
        }
    }
};

// Four CTAs an SM leave 64 registers, and three of the four kernels for bf16 parameters with 8-bit states then keep up
// to 6 words in local memory.  With three CTAs and 80 registers none does, and they are slower: 100 million
// parameters with bf16 gradients 266 -> 289 us, with fp32 ones 268 -> 289, with a master 281 -> 301 and 298 -> 309.
template <class P, class G, bool kState8, bool kMaster, int kCap>
__global__ void __launch_bounds__(kWarps * 32, 4) dg_adamw_kernel(const __grid_constant__ Args<kCap> a) {
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

    Step s{a.b1, a.b2, a.one_minus_b1, a.one_minus_b2, a.eps, -a.step_size, a.inv_root_bc2, t.decay, a.grad_scale,
           a.step, a.first_tensor + lo, a.stochastic};
    if (a.grad_scale_dev) s.gscale *= *a.grad_scale_dev;
    if (a.step_dev || a.lr_dev) {
        __shared__ float shared[3];
        if (a.step_dev) s.step = static_cast<uint32_t>(*a.step_dev);
        if (threadIdx.x == 0) {
            const double lr = a.lr_dev ? static_cast<double>(*a.lr_dev) : a.lr;
            // 1 - b^t without cancellation; b = 0 gives 1
            const double c1 = a.beta1 > 0 ? -expm1(s.step * log(a.beta1)) : 1.0;
            const double c2 = a.beta2 > 0 ? -expm1(s.step * log(a.beta2)) : 1.0;
            shared[0] = static_cast<float>(-lr / c1);
            shared[1] = static_cast<float>(1.0 / sqrt(c2));
            shared[2] = static_cast<float>(1.0 - lr * static_cast<double>(t.decay));
        }
        __syncthreads();
        s.rate = shared[0];
        s.bias = shared[1];
        s.keep = shared[2];
    }

    // This warp's blocks are consecutive, so that their addresses differ by constants.
    const long long n = t.n;
    const int first_own = warp * a.blocks_per_warp;
    const long long base = (static_cast<long long>(cta - a.first_cta[lo]) * kWarps * a.blocks_per_warp + first_own) * kBlock;
    const int blocks = static_cast<int>(min(static_cast<long long>(a.blocks_per_warp), (n - base + kBlock - 1) / kBlock));
    const int whole = t.aligned ? static_cast<int>(min(static_cast<long long>(blocks), (n - base) / kBlock)) : 0;
    // A CTA's exponents are read before any is written and written together at the end: read and written one
    // by one, each read waited for the neighbours' writes to the same 32-byte sector (1.07 ms instead of
    // 0.43 ms for 120 million bf16 parameters).
    __shared__ int8_t exps[2][kWarps * kMaxBlocksPerWarp];
    const long long first_block = static_cast<long long>(cta - a.first_cta[lo]) * a.blocks_per_warp * kWarps;
    const int k = threadIdx.x;
    const bool mine = k < a.blocks_per_warp * kWarps && (first_block + k) * kBlock < n;
    if constexpr (kState8) {
        if (mine) {
            exps[0][k] = t.m_exp[first_block + k];
            exps[1][k] = t.v_exp[first_block + k];
        }
        __syncthreads();
    }
    const Bases<P, G, kState8> from(t, base + lane * 8);
#pragma unroll 1
    for (int k = 0; k < blocks; ++k) {
        Lane<P, G, kState8, kMaster> x;
        int em = 0, ev = 0;
        if constexpr (kState8) {
            em = exps[0][first_own + k];
            ev = exps[1][first_own + k];
        }
        if (k < whole) {
            x.template load<true>(from, k * kBlock, 8);
            x.template update<true>(from, s, a.keys, k * kBlock, 8, em, ev);
        } else {
            const long long left = n - (base + k * kBlock + lane * 8);
            const int live = left <= 0 ? 0 : (left < 8 ? static_cast<int>(left) : 8);
            x.template load<false>(from, k * kBlock, live);
            x.template update<false>(from, s, a.keys, k * kBlock, live, em, ev);
        }
        if constexpr (kState8) {
            __syncwarp();
            if (lane == 0) {
                exps[0][first_own + k] = static_cast<int8_t>(em);
                exps[1][first_own + k] = static_cast<int8_t>(ev);
            }
        }
    }
    if constexpr (kState8) {
        __syncthreads();
        if (mine) {
            t.m_exp[first_block + k] = exps[0][k];
            t.v_exp[first_block + k] = exps[1][k];
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

// Launch the tensors [begin, end) as one grid (none where all are empty).
template <int kCap>
dg_status launch_range(const dg_adamw_params* p, const dg_adamw_tensor* tensors, int begin, int end,
                       int blocks_per_warp, bool master, int* launches, cudaStream_t s) {
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
    for (uint32_t r = 0; r < 10; ++r) {
        a.keys.k[r][0] = static_cast<uint32_t>(p->seed) + r * 0x9E3779B9u;
        a.keys.k[r][1] = static_cast<uint32_t>(p->seed >> 32) + r * 0xBB67AE85u;
    }
    a.step = static_cast<uint32_t>(p->step);
    a.first_tensor = static_cast<uint32_t>(begin);
    a.stochastic = p->stochastic;
    a.blocks_per_warp = blocks_per_warp;
    a.n_tensors = end - begin;
    const long long per_cta = static_cast<long long>(kBlock) * kWarps * blocks_per_warp;
    long long ctas = 0;
    const uintptr_t pa = p->param_type == DG_FP32 ? 32 : 16, ga = p->grad_type == DG_FP32 ? 32 : 16;
    const uintptr_t sa = p->state_bits == 8 ? 8 : 32;
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
        t.decay = p->lr_dev || p->step_dev
                      ? x.weight_decay
                      : static_cast<float>(1.0 - p->lr * static_cast<double>(x.weight_decay));
        t.aligned = !(misaligned(x.param, pa) || misaligned(x.grad, ga) || misaligned(x.m, sa) ||
                      misaligned(x.v, sa) || misaligned(x.master, 32));
        a.first_cta[i - begin] = static_cast<int>(ctas);
        ctas += (x.n + per_cta - 1) / per_cta;
        if (ctas > 0x7fffffffLL) return DG_EINVAL;   // over 2^42 elements
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
    if (e != cudaSuccess) return DG_ECUDA;
    ++*launches;
    return DG_OK;
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
    if (p->eps > 0 && p->eps < 0x1p-126) return DG_EINVAL;      // div_sfu takes a subnormal for 0
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
    bool any_master = false;
    for (int i = 0; i < n_tensors; ++i) {
        const dg_adamw_tensor& x = tensors[i];
        if (x.n < 0 || x.n >= (1LL << 34)) return DG_EINVAL;     // element / 4 is one counter word
        if (!std::isfinite(x.weight_decay)) return DG_EINVAL;
        any_master = any_master || x.master;
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
    // a master copy for all tensors of a call or for none, and only beside bf16 parameters that it rounds to (an
    // empty tensor needs none, but one that names it speaks for the call)
    if (any_master && (with_master != live || p->param_type != DG_BF16 || p->stochastic)) return DG_EINVAL;
    // 8-bit states of many elements: 8 blocks a warp, which share the search of the list, the constants and the
    // exponents' accesses (262144 x 2816 bf16 parameters: 1.86 ms with 8, 1.92 with 4, 2.25 with 1).  fp32 states
    // (bound by the bytes; 65536 x 2816 with master: 0.751 ms with 1, 0.799 with 8) and few elements (to spread
    // them over the SMs): one.
    const int sms = device_sm_count();
    if (sms <= 0) return DG_ECUDA;
    const bool many = total > static_cast<long long>(sms) * 8 * kWarps * kBlock * kMaxBlocksPerWarp;
    const int bpw = p->state_bits == 8 && many ? kMaxBlocksPerWarp : 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int launches = 0;
    for (int begin = 0; begin < n_tensors;) {
        const int left = n_tensors - begin;
        const int end = begin + (left > kManyTensors ? kManyTensors : left);
        const dg_status st =
            left <= kFewTensors ? launch_range<kFewTensors>(p, tensors, begin, end, bpw, any_master, &launches, s)
                                : launch_range<kManyTensors>(p, tensors, begin, end, bpw, any_master, &launches, s);
        if (st != DG_OK) return st;
        begin = end;
    }
    set_last_launches(launches);
    return DG_OK;
}

}  // extern "C"
