// act8_grad.cu -- weight gradients of linear layers from 8-bit activation
// checkpoints: G = beta G + (dY^T X^) diag(gain) + dy_sum shift^T.
//
// First form: CUDA cores, fp32, one 64 x 64 tile of G per block, 16 tokens at a
// time through shared memory.
#include <algorithm>
#include <cmath>

#include "act8.cuh"
#include "gemm.h"

namespace muon {

namespace {

constexpr int kT = 64, kKT = 16;

__global__ void __launch_bounds__(256) act8_grad_simple(muon_act8_grad_item I, int dy_dt, int w_dt) {
    __shared__ float sd[kKT][kT + 4], sx[kKT][kT + 4];
    const int o0 = blockIdx.y * kT, i0 = blockIdx.x * kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int t0 = 0; t0 < I.c.rows; t0 += kKT) {
        for (int k = threadIdx.x; k < kKT * kT; k += 256) {
            const int r = k / kT, c = k % kT;
            const long long t = t0 + r;
            const bool in = t < I.c.rows;
            sd[r][c] = in && o0 + c < I.out ? ld_elem(I.dY, t * I.lddy + o0 + c, dy_dt) : 0.f;
            float x = 0.f;
            if (in && i0 + c < I.c.cols) {
                const int b = I.c.e[t * I.c.lde + (i0 + c) / kActBlock];
                x = (float)I.c.q[t * I.c.ldq + i0 + c] * (b == kActBad ? __uint_as_float(0x7FC00000u) : act8_scale(b));
                if (dy_dt == DT_FP16) x = __half2float(__float2half_rn(x));
            }
            sx[r][c] = x;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKT; ++k)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sd[k][ty * 4 + a], sx[k][tx * 4 + b], acc[a][b]);
        __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int o = o0 + ty * 4 + a, c = i0 + tx * 4 + b;
            if (o >= I.out || c >= I.c.cols) continue;
            const long long at = (long long)o * I.c.cols + c;
            float g = acc[a][b];
            if (I.gain) g *= ld_elem(I.gain, c, w_dt);
            if (I.shift) g = fmaf(I.dy_sum[o], ld_elem(I.shift, c, w_dt), g);
            if (I.beta != 0.f) g = fmaf(I.beta, ld_elem(I.G, at, w_dt), g);
            st_elem(I.G, at, w_dt, g);
        }
}

bool valid(int dt) { return dt == DT_BF16 || dt == DT_FP16 || dt == DT_FP32; }

muon_status check_items(const muon_act8_grad_item* items, int n) {
    if (!items || n < 1) return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const muon_act8_grad_item& q = items[i];
        if (!act8_valid(q.c) || q.out < 1 || q.lddy < q.out || !q.G || (q.c.rows > 0 && !q.dY) ||
            !q.shift != !q.dy_sum || !std::isfinite(q.beta))
            return MUON_ERR_INVALID_ARG;
    }
    return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status act8_grad_workspace_size(const muon_act8_grad_item* items, int n, muon_dtype dy_dtype, size_t* bytes) {
    if (!bytes || !valid(dy_dtype)) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_items(items, n);
    if (st != MUON_OK) return st;
    *bytes = 0;
    return MUON_OK;
}

muon_status act8_grad_batched(const muon_act8_grad_item* items, int n, muon_dtype dy_dtype, muon_dtype w_dtype,
                              void* workspace, size_t ws_bytes, int* d_status, muon_stream_t stream) {
    (void)workspace; (void)ws_bytes; (void)d_status;
    if (!valid(dy_dtype) || !valid(w_dtype)) return MUON_ERR_INVALID_ARG;
    muon_status st = check_items(items, n);
    if (st != MUON_OK) return st;
    st = check_device();
    if (st != MUON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int i = 0; i < n; ++i) {
        const muon_act8_grad_item& q = items[i];
        const dim3 grid((q.c.cols + kT - 1) / kT, (q.out + kT - 1) / kT);
        trace_begin(MUON_KERNEL_ACT8_GRAD, 2.0 * q.c.rows * q.out * q.c.cols, s);
        act8_grad_simple<<<grid, 256, 0, s>>>(q, dy_dtype, w_dtype);
        trace_end(s);
        if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
    }
    return MUON_OK;
}

}  // extern "C"
