// adamw.cu -- AdamW over many tensors in one launch, with first and second moments in fp32 or in
// 8 bits, and the gradient norm that clips it.
//
//   g' = s g                                     s: a device scalar (clipping, loss scaling)
//   m  = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit states keep m and r = sqrt(v) (half of v's range in powers of two, and what the update
// divides by), each in blocks of 32 elements under one power-of-two scale (an E8M0 byte b for
// 2^(b - 127); b = 0: a block of zeros; b = 0xFF: the block held NaN or Inf):
//   m  E4M3 codes, the smallest scale that keeps the block's largest |m| at 448 or below;
//   r  code c > 0 for (1 + (c & 15) / 16) 2^((c >> 4) - 15), code 0 for 0; the scale keeps the
//      largest r at 31/16 or below.  No sign to store, so one more mantissa bit than E4M3; a
//      positive r below the smallest code takes the smallest code, so the update never divides
//      by a second moment that rounding made zero.
// Both round stochastically: with b2 = 0.999 a step changes r by less than 0.05 %, far below half
// a code (3 %), so rounding to nearest would leave it where it is for ever; floor(x + u) with u
// uniform keeps the mean exact to 2^-16 of a code.  u comes from a hash of (seed, t, position),
// so a step is a function of its inputs.  bf16 parameters may be rounded the same way.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "quant_common.cuh"
#include "mxmoe_internal.h"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                        // consecutive elements of a thread
constexpr int kChunk = kThreads * kPer;        // elements of a chunk: the unit a CTA works on
constexpr int kNormCtas = 1216;                // most CTAs of the norm: 8 on each of 152 SMs

// One tensor of the plan in device memory.
struct Slot {
    void* p;
    const void* g;
    void* m;
    void* v;            // fp32: v; 8 bits: codes of r
    uint8_t* sm;
    uint8_t* sr;
    void* copy;         // bf16 copy of an fp32 parameter, or null
    int64_t n;
    int64_t chunk0;     // first chunk of the tensor in the plan
    int64_t pos0;       // position of its first element: tensors start at multiples of 32
    float wd, lr_mult;
    int32_t p_f32, g_f32;
};

// The plan: header, slots, then for every chunk the index of its tensor.
struct Header {
    unsigned int step_done, norm_done;   // CTAs that have finished (back to 0 at the end of a call)
    unsigned int pad[14];
    double partial[kNormCtas];
};

struct PlanView {
    Header* h;
    const Slot* slots;
    const int32_t* of_chunk;
};

__host__ __device__ inline PlanView view(void* plan, int n) {
    PlanView v;
    v.h = static_cast<Header*>(plan);
    v.slots = reinterpret_cast<const Slot*>(static_cast<char*>(plan) + sizeof(Header));
    v.of_chunk = reinterpret_cast<const int32_t*>(v.slots + n);
    return v;
}

// ------------------------------------------------------------------ random bits
// Multiply, shift, multiply, shift: a bijection of 32-bit words whose output bits all depend on
// every input bit above half way; the constants are odd and otherwise free.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x *= 0x9E3779B1u;
    x ^= x >> 15;
    x *= 0x85EBCA77u;
    return x ^ (x >> 13);
}

// Key of the elements whose position has the upper word hi, in step t.
__device__ __forceinline__ uint32_t step_key(uint32_t seed, int64_t t) {
    return mix(seed + 0x9E3779B9u * static_cast<uint32_t>(t)) ^ static_cast<uint32_t>(static_cast<uint64_t>(t) >> 32);
}

// ------------------------------------------------------------------ values of 8 elements
struct Vals {
    float x[kPer];
};

__device__ __forceinline__ void load_f32(const float* src, int valid, float (&x)[kPer]) {
    if (valid == kPer) {
        const uint4 a = *reinterpret_cast<const uint4*>(src), b = *reinterpret_cast<const uint4*>(src + 4);
        x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
        x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = i < valid ? src[i] : 0.f;
    }
}

__device__ __forceinline__ void load_bf16(const uint16_t* src, int valid, float (&x)[kPer]) {
    if (valid == kPer) {
        const uint4 a = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = i < valid ? __uint_as_float(static_cast<uint32_t>(src[i]) << 16) : 0.f;
    }
}

__device__ __forceinline__ void store_f32(float* dst, int valid, const float (&x)[kPer]) {
    if (valid == kPer) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < valid) dst[i] = x[i];
    }
}

__device__ __forceinline__ void store_words(uint16_t* dst, int valid, const uint32_t (&w)[4]) {   // 8 bf16
    if (valid == kPer) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < valid) dst[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

__device__ __forceinline__ void load_bytes(const uint8_t* src, int valid, uint32_t (&w)[2]) {
    if (valid == kPer) {
        const uint2 a = *reinterpret_cast<const uint2*>(src);
        w[0] = a.x;
        w[1] = a.y;
    } else {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < valid) w[i / 4] |= static_cast<uint32_t>(src[i]) << (8 * (i & 3));
    }
}

__device__ __forceinline__ void store_bytes(uint8_t* dst, int valid, const uint32_t (&w)[2]) {
    if (valid == kPer) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i < valid) dst[i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ void load_any(const void* base, bool f32, int64_t at, int valid, float (&x)[kPer]) {
    if (f32) load_f32(static_cast<const float*>(base) + at, valid, x);
    else load_bf16(static_cast<const uint16_t*>(base) + at, valid, x);
}

// ------------------------------------------------------------------ 8-bit states
// 2^(b - 127); 0 for b = 0 (a block of zeros), Inf for b = 0xFF (times a NaN or zero code: NaN)
__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float(b << 23); }

__device__ __forceinline__ void decode_m(const uint32_t (&w)[2], uint32_t b, float (&x)[kPer]) {
    const float s = scale_value(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t two = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        float lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(lo), "=f"(hi) : "r"(h));
        x[2 * i] = lo * s;
        x[2 * i + 1] = hi * s;
    }
}

__device__ __forceinline__ void decode_r(const uint32_t (&w)[2], uint32_t b, float (&x)[kPer]) {
    const float s = scale_value(b);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t c = (w[i / 4] >> (8 * (i & 3))) & 0xFFu;
        x[i] = (c != 0 ? __uint_as_float((c << 19) + (112u << 23)) : 0.f) * s;
    }
}

// Largest of the 32 elements' magnitude bits: 8 of this thread, 8 of each of its three neighbours.
// As integers NaN > Inf > every finite value, so none is lost.
__device__ __forceinline__ uint32_t block_amax(const float (&x)[kPer]) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    return max(a, __shfl_xor_sync(0xffffffffu, a, 2));
}

// Scale byte for a block whose largest magnitude has the bits a: exponent minus `shift`, one more
// where the mantissa passes `over` (the code's largest one).  1 at least for a block with a
// nonzero value, so that 0 stays the block of zeros.
__device__ __forceinline__ uint32_t block_byte(uint32_t a, int shift, uint32_t over) {
    if (a >= 0x7F800000u) return 0xFFu;
    if (a == 0) return 0;
    const int b = static_cast<int>(a >> 23) - shift + ((a & 0x7FFFFFu) > over ? 1 : 0);
    return b < 1 ? 1u : static_cast<uint32_t>(b);
}

// E4M3 codes of x / 2^(b - 127), stochastically rounded by 16 bits of u each: the 20 bits below
// the code's 3 mantissa bits are filled up by u, then cut.  Below 2^-6 the code's grid is 2^-9
// throughout; adding 2^-6 first gives fp32 that grid.
__device__ __forceinline__ void encode_m(const float (&x)[kPer], uint32_t b, const uint32_t (&u)[kPer], uint32_t (&w)[2]) {
    if (b == 0xFFu) {
        w[0] = w[1] = 0x7F7F7F7Fu;
        return;
    }
    const float inv = __uint_as_float((254u - (b == 0 ? 1u : b)) << 23);
    float q[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        float y = fabsf(x[i]) * inv;
        const bool small = y < 0.015625f;
        if (small) y += 0.015625f;
        y = __uint_as_float((__float_as_uint(y) + ((u[i] >> 16) << 4)) & ~0xFFFFFu);
        if (small) y -= 0.015625f;
        q[i] = copysignf(y, x[i]);
    }
    w[0] = cvt_e4m3x4(q[0], q[1], q[2], q[3]);
    w[1] = cvt_e4m3x4(q[4], q[5], q[6], q[7]);
}

__device__ __forceinline__ void encode_r(const float (&r)[kPer], uint32_t b, const uint32_t (&u)[kPer], uint32_t (&w)[2]) {
    w[0] = w[1] = 0;
    if (b == 0xFFu) return;
    const float inv = __uint_as_float((254u - (b == 0 ? 1u : b)) << 23);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t bits = __float_as_uint(r[i] * inv) + ((u[i] & 0xFFFFu) << 3);
        const int c = static_cast<int>(bits >> 19) - (112 << 4);
        w[i / 4] |= (r[i] > 0.f ? static_cast<uint32_t>(c < 1 ? 1 : c) : 0u) << (8 * (i & 3));
    }
}

// ------------------------------------------------------------------ the step
struct StepArgs {
    int n;
    int64_t chunks;
    int64_t* step;
    double log_b1, log_b2;   // ln b1, ln b2
    float lr, b1, c1, b2, c2, eps;   // c1 = 1 - b1, c2 = 1 - b2, each rounded from 64 bits
    const float* lr_dev;
    const float* grad_scale;
    uint32_t seed;
    int stochastic;
};

template <bool EIGHT>
__global__ void __launch_bounds__(kThreads) adamw_step_kernel(void* plan, const StepArgs a) {
    const PlanView pv = view(plan, a.n);
    __shared__ float s_bc[2];
    const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
    const int64_t t = *a.step + 1;
    if (!isfinite(gs)) return;   // the gradients were not finite: the step is skipped, t stays
    if (threadIdx.x == 0) {
        s_bc[0] = -expm1f(static_cast<float>(static_cast<double>(t) * a.log_b1));            // 1 - b1^t
        s_bc[1] = rsqrtf(-expm1f(static_cast<float>(static_cast<double>(t) * a.log_b2)));   // (1 - b2^t)^-1/2
    }
    __syncthreads();
    const int64_t chunk = blockIdx.x;
    const Slot& sl = pv.slots[pv.of_chunk[chunk]];
    const int64_t at = (chunk - sl.chunk0) * kChunk + threadIdx.x * kPer;
    const int64_t left = sl.n - at;
    const int valid = left >= kPer ? kPer : (left > 0 ? static_cast<int>(left) : 0);
    const float lr = (a.lr_dev != nullptr ? *a.lr_dev : a.lr) * sl.lr_mult;
    const float keep = 1.0f - lr * sl.wd, lr_t = lr / s_bc[0], inv_v = s_bc[1];
    float p[kPer], g[kPer], m[kPer], v[kPer], r[kPer];
    uint32_t wm[2], wr[2];
    load_any(sl.p, sl.p_f32, at, valid, p);
    load_any(sl.g, sl.g_f32, at, valid, g);
    if (EIGHT) {
        load_bytes(static_cast<const uint8_t*>(sl.m) + at, valid, wm);
        load_bytes(static_cast<const uint8_t*>(sl.v) + at, valid, wr);
        decode_m(wm, valid > 0 ? sl.sm[at / 32] : 0u, m);
        decode_r(wr, valid > 0 ? sl.sr[at / 32] : 0u, r);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = r[i] * r[i];
    } else {
        load_f32(static_cast<const float*>(sl.m) + at, valid, m);
        load_f32(static_cast<const float*>(sl.v) + at, valid, v);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float x = g[i] * gs;
        m[i] = fmaf(a.b1, m[i], a.c1 * x);
        v[i] = fmaf(a.b2, v[i], a.c2 * x * x);
        r[i] = sqrtf(v[i]);
        p[i] = fmaf(p[i], keep, -lr_t * (m[i] / fmaf(r[i], inv_v, a.eps)));
    }
    const bool sr_p = a.stochastic && !sl.p_f32;
    uint32_t u[kPer];
    if (EIGHT || sr_p) {
        const uint64_t pos = static_cast<uint64_t>(sl.pos0 + at);
        const uint32_t key = mix(step_key(a.seed, t) + static_cast<uint32_t>(pos >> 32));
#pragma unroll
        for (int i = 0; i < kPer; ++i) u[i] = mix((static_cast<uint32_t>(pos) + i) ^ key);
    }
    if (sl.p_f32) {
        store_f32(static_cast<float*>(sl.p) + at, valid, p);
        if (sl.copy != nullptr) {
            const uint32_t w[4] = {pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7])};
            store_words(static_cast<uint16_t*>(sl.copy) + at, valid, w);
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sr_p) {
                uint32_t h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t x = u[2 * i + j];
                    const uint32_t y = ((x ^ (x >> 7)) * 0xC2B2AE3Du) >> 16;
                    const uint32_t bits = __float_as_uint(p[2 * i + j]);
                    h[j] = (bits & 0x7F800000u) == 0x7F800000u ? bits | ((bits & 0x7FFFFFu) != 0 ? 0x400000u : 0u) : bits + y;
                }
                w[i] = __byte_perm(h[0], h[1], 0x7632);
            } else {
                w[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
            }
        }
        store_words(static_cast<uint16_t*>(sl.p) + at, valid, w);
    }
    if (EIGHT) {
        const uint32_t bm = block_byte(block_amax(m), 8, 0x600000u), br = block_byte(block_amax(r), 0, 0x780000u);
        encode_m(m, bm, u, wm);
        encode_r(r, br, u, wr);
        store_bytes(static_cast<uint8_t*>(sl.m) + at, valid, wm);
        store_bytes(static_cast<uint8_t*>(sl.v) + at, valid, wr);
        if ((threadIdx.x & 3) == 0 && valid > 0) {
            sl.sm[at / 32] = static_cast<uint8_t>(bm);
            sl.sr[at / 32] = static_cast<uint8_t>(br);
        }
    } else {
        store_f32(static_cast<float*>(sl.m) + at, valid, m);
        store_f32(static_cast<float*>(sl.v) + at, valid, v);
    }
    // every CTA has read the step by now: the last to arrive here counts it
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&pv.h->step_done, 1u) == gridDim.x - 1) {
            pv.h->step_done = 0;
            *a.step = t;
        }
    }
}

// ------------------------------------------------------------------ the gradient norm
// Squares are summed in fp32 over a thread's 8 elements of a chunk and in 64 bits above that, in a
// fixed order: per thread over its chunks, per warp and CTA by a tree, over the CTAs in order.
__global__ void __launch_bounds__(kThreads) adamw_norm_kernel(void* plan, int n, int64_t chunks, float max_norm,
                                                              float* out) {
    const PlanView pv = view(plan, n);
    __shared__ double s_sum[kThreads / 32];
    __shared__ bool s_last;
    double sum = 0.0;
    for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const Slot& sl = pv.slots[pv.of_chunk[chunk]];
        const int64_t at = (chunk - sl.chunk0) * kChunk + threadIdx.x * kPer;
        const int64_t left = sl.n - at;
        const int valid = left >= kPer ? kPer : (left > 0 ? static_cast<int>(left) : 0);
        float g[kPer];
        load_any(sl.g, sl.g_f32, at, valid, g);
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) part = fmaf(g[i], g[i], part);
        sum += static_cast<double>(part);
    }
    auto block_sum = [&](double x) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
        __syncthreads();
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) total += s_sum[w];
        return total;
    };
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        pv.h->partial[blockIdx.x] = sum;
        __threadfence();
        s_last = atomicAdd(&pv.h->norm_done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double x = 0.0;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) x += __ldcg(&pv.h->partial[i]);
    x = block_sum(x);
    if (threadIdx.x == 0) {
        pv.h->norm_done = 0;
        const double norm = sqrt(x);
        out[0] = static_cast<float>(norm);
        // a norm that is not finite gives NaN, which adamw_step takes as "skip this step"
        out[1] = !isfinite(norm) ? __uint_as_float(0x7FC00000u)
                 : max_norm > 0.f && norm > max_norm ? static_cast<float>(max_norm / norm) : 1.0f;
    }
}

// ------------------------------------------------------------------ the states' values
__global__ void __launch_bounds__(kThreads) adamw_values_kernel(void* plan, int n, uint16_t* mom, uint16_t* root) {
    const PlanView pv = view(plan, n);
    const int64_t chunk = blockIdx.x;
    const Slot& sl = pv.slots[pv.of_chunk[chunk]];
    const int64_t at = (chunk - sl.chunk0) * kChunk + threadIdx.x * kPer;
    const int64_t left = sl.n - at;
    const int valid = left >= kPer ? kPer : (left > 0 ? static_cast<int>(left) : 0);
    if (valid == 0) return;
    uint32_t w[2];
    float x[kPer];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        load_bytes(static_cast<const uint8_t*>(which ? sl.v : sl.m) + at, valid, w);
        if (which) decode_r(w, sl.sr[at / 32], x);
        else decode_m(w, sl.sm[at / 32], x);
        const uint32_t o[4] = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
        store_words((which ? root : mom) + sl.pos0 + at, valid, o);
    }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count() {
    static int count[64] = {0};
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (count[dev] == 0 && cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return count[dev];
}

}  // namespace

int build_adamw_plan(const adamw_tensor* tensors, int n, int state_bits, void* image, size_t image_bytes, adamw_info* info) {
    const bool eight = state_bits == 8;
    int64_t chunks = 0, pos = 0;
    for (int i = 0; i < n; ++i) {
        const adamw_tensor& x = tensors[i];
        if (x.n < 1 || x.n >= (int64_t(1) << 40)) return MX_ERR_INVALID_ARG;
        if (!x.param || !x.grad || !x.moment || !x.second) return MX_ERR_INVALID_ARG;
        if (eight != (x.scale_m != nullptr) || eight != (x.scale_r != nullptr)) return MX_ERR_INVALID_ARG;
        if ((x.param_dtype != MX_DTYPE_BF16 && x.param_dtype != MX_DTYPE_F32) ||
            (x.grad_dtype != MX_DTYPE_BF16 && x.grad_dtype != MX_DTYPE_F32))
            return MX_ERR_INVALID_ARG;
        if (x.copy != nullptr && x.param_dtype != MX_DTYPE_F32) return MX_ERR_INVALID_ARG;
        if (!std::isfinite(x.weight_decay) || x.weight_decay < 0.f || !std::isfinite(x.lr_mult) || x.lr_mult < 0.f)
            return MX_ERR_INVALID_ARG;
        if (!aligned16(x.param) || !aligned16(x.grad) || !aligned16(x.moment) || !aligned16(x.second) || !aligned16(x.copy))
            return MX_ERR_ALIGNMENT;
        chunks += ceil_div(x.n, kChunk);
        pos += round_up(x.n, 32);
    }
    if (chunks >= (int64_t(1) << 31)) return MX_ERR_UNSUPPORTED;
    info->positions = pos;
    info->chunks = chunks;
    info->tensors = n;
    info->state_bits = state_bits;
    info->bytes = static_cast<int64_t>(round_up(sizeof(Header) + n * sizeof(Slot) + chunks * sizeof(int32_t), 16));
    if (image == nullptr) return MX_OK;
    if (image_bytes < static_cast<size_t>(info->bytes)) return MX_ERR_INVALID_ARG;
    auto* h = static_cast<Header*>(image);
    *h = Header{};
    auto* slots = reinterpret_cast<Slot*>(static_cast<char*>(image) + sizeof(Header));
    auto* of_chunk = reinterpret_cast<int32_t*>(slots + n);
    chunks = pos = 0;
    for (int i = 0; i < n; ++i) {
        const adamw_tensor& x = tensors[i];
        slots[i] = Slot{x.param, x.grad, x.moment, x.second, x.scale_m, x.scale_r, x.copy, x.n, chunks, pos, x.weight_decay,
                        x.lr_mult, x.param_dtype == MX_DTYPE_F32, x.grad_dtype == MX_DTYPE_F32};
        for (int64_t c = 0; c < ceil_div(x.n, kChunk); ++c) of_chunk[chunks++] = i;
        pos += round_up(x.n, 32);
    }
    return MX_OK;
}

int launch_adamw_step(void* plan, const adamw_info& info, int64_t* step, double lr, double beta1, double beta2, double eps,
                      const float* lr_dev, const float* grad_scale, uint32_t seed, bool stochastic, cudaStream_t stream) {
    StepArgs a;
    a.n = info.tensors;
    a.chunks = info.chunks;
    a.step = step;
    a.log_b1 = std::log(beta1);   // b1 = 0: -inf, and 1 - b1^t = 1
    a.log_b2 = std::log(beta2);
    a.lr = static_cast<float>(lr);
    a.b1 = static_cast<float>(beta1);
    a.c1 = static_cast<float>(1.0 - beta1);
    a.b2 = static_cast<float>(beta2);
    a.c2 = static_cast<float>(1.0 - beta2);
    a.eps = static_cast<float>(eps);
    a.lr_dev = lr_dev;
    a.grad_scale = grad_scale;
    a.seed = seed;
    a.stochastic = stochastic;
    const unsigned grid = static_cast<unsigned>(info.chunks);
    if (info.state_bits == 8) adamw_step_kernel<true><<<grid, kThreads, 0, stream>>>(plan, a);
    else adamw_step_kernel<false><<<grid, kThreads, 0, stream>>>(plan, a);
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

int launch_adamw_norm(void* plan, const adamw_info& info, double max_norm, float* out, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return MX_ERR_CUDA;
    int64_t grid = static_cast<int64_t>(sms) * 8;
    grid = grid > kNormCtas ? kNormCtas : grid;
    grid = grid > info.chunks ? info.chunks : grid;
    adamw_norm_kernel<<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(plan, info.tensors, info.chunks,
                                                                            static_cast<float>(max_norm), out);
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

int launch_adamw_values(void* plan, const adamw_info& info, void* moment, void* root, cudaStream_t stream) {
    adamw_values_kernel<<<static_cast<unsigned>(info.chunks), kThreads, 0, stream>>>(
        plan, info.tensors, static_cast<uint16_t*>(moment), static_cast<uint16_t*>(root));
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

}  // namespace mx
