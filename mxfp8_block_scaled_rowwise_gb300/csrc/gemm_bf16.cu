// gemm_bf16.cu -- expert grouped products on bf16 operands with ragged groups:
//   forward  C[r]  = bf16( A[r] W_e^T )            rows r in [off[e], off[e + 1])
//   dgrad    dX[r] = bf16( dY[r] W_e )
//   wgrad    dW[e] = sum over the expert's rows of dY[r]^T X[r]   (fp32; zeros without rows)
// fp32 accumulation.  One CTA per 64 x 64 output tile, operands through shared memory as fp32,
// every index checked against the expert's own extent.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxmoe_internal.h"

namespace mx {
namespace {

constexpr int kTile = 64;
constexpr int kDepth = 16;
constexpr int kThreads = 256;
constexpr int kFwd = kBf16Fwd, kDgrad = kBf16Dgrad, kWgrad = kBf16Wgrad;

__device__ bool offsets_ok(const int32_t* off, int E, int64_t R) {
    bool bad = false;
    for (int e = threadIdx.x; e < E; e += kThreads) bad |= off[e + 1] < off[e];
    if (threadIdx.x == 0) bad |= off[0] != 0 || off[E] > R;
    return !__syncthreads_or(bad);
}

template <int PASS>
__global__ void __launch_bounds__(kThreads) grouped_bf16_kernel(const __nv_bfloat16* A, const __nv_bfloat16* B,
                                                                const int32_t* off, int E, int64_t R, int64_t N,
                                                                int64_t K, void* out, int* dev_err) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    if (!offsets_ok(off, E, R)) {
        if (threadIdx.x == 0) atomicOr(dev_err, MX_DEVERR_BAD_SEGMENTS);
        return;
    }
    int e = 0;
    int64_t m0 = 0;   // first output row of the tile: within the expert's rows, or within N (wgrad)
    if (PASS == kWgrad) {
        const int64_t mt = (N + kTile - 1) / kTile;
        e = static_cast<int>(blockIdx.y / mt);
        m0 = (blockIdx.y - e * mt) * kTile;
    } else {
        int64_t left = blockIdx.y;
        for (; e < E; ++e) {
            const int64_t t = (static_cast<int64_t>(off[e + 1]) - off[e] + kTile - 1) / kTile;
            if (left < t) break;
            left -= t;
        }
        if (e == E) return;
        m0 = left * kTile;
    }
    const int64_t r0 = off[e], rows = static_cast<int64_t>(off[e + 1]) - r0;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int64_t M = PASS == kWgrad ? N : rows, cols = PASS == kWgrad ? K : N, depth = PASS == kWgrad ? rows : K;
    float acc[4][4] = {};
    const int tm = threadIdx.x / 16 * 4, tn = threadIdx.x % 16 * 4;
    for (int64_t k0 = 0; k0 < depth; k0 += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
            const int x = PASS == kWgrad ? i % kTile : i / kDepth, k = PASS == kWgrad ? i / kTile : i % kDepth;
            const bool in = m0 + x < M && k0 + k < depth;
            sa[k][x] = in ? __bfloat162float(PASS == kWgrad ? A[(r0 + k0 + k) * N + m0 + x] : A[(r0 + m0 + x) * K + k0 + k]) : 0.f;
        }
        for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
            const int x = PASS == kFwd ? i / kDepth : i % kTile, k = PASS == kFwd ? i % kDepth : i / kTile;
            const bool in = n0 + x < cols && k0 + k < depth;
            const int64_t at = PASS == kFwd ? (e * N + n0 + x) * K + k0 + k
                               : PASS == kDgrad ? (e * K + k0 + k) * N + n0 + x : (r0 + k0 + k) * K + n0 + x;
            sb[k][x] = in ? __bfloat162float(B[at]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][tm + i], sb[k][tn + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            if (m0 + tm + i >= M || n0 + tn + j >= cols) continue;
            const int64_t at = ((PASS == kWgrad ? e * N : r0) + m0 + tm + i) * cols + n0 + tn + j;
            if (PASS == kWgrad) static_cast<float*>(out)[at] = acc[i][j];
            else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(acc[i][j]);
        }
}

}  // namespace

int launch_grouped_gemm_bf16(int pass, const void* A, const void* B, const int32_t* off, int E, int64_t R, int64_t N,
                             int64_t K, void* out, int* dev_err, cudaStream_t stream) {
    const int64_t mt = pass == kWgrad ? E * ceil_div(N, kTile) : R / kTile + E, nt = ceil_div(pass == kWgrad ? K : N, kTile);
    if (mt > 65535 || nt >= (int64_t(1) << 31)) return MX_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(nt), static_cast<unsigned>(mt));
    const auto* a = static_cast<const __nv_bfloat16*>(A);
    const auto* b = static_cast<const __nv_bfloat16*>(B);
    if (pass == kFwd) grouped_bf16_kernel<kFwd><<<grid, kThreads, 0, stream>>>(a, b, off, E, R, N, K, out, dev_err);
    else if (pass == kDgrad) grouped_bf16_kernel<kDgrad><<<grid, kThreads, 0, stream>>>(a, b, off, E, R, N, K, out, dev_err);
    else grouped_bf16_kernel<kWgrad><<<grid, kThreads, 0, stream>>>(a, b, off, E, R, N, K, out, dev_err);
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

}  // namespace mx
