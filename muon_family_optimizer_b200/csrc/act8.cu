// act8.cu -- writing and reading 8-bit activation checkpoints (act8.cuh has the
// format).
//
// Both passes are bound by HBM: 2 + 1 + 1/32 bytes per element for 16-bit
// data.  A warp takes four rows of a 256-column segment, eight columns per lane
// (16-byte loads of 16-bit data, 8-byte accesses of codes), every load issued
// before any use; a block's four lanes find its exponent with two shuffles.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "act8.cuh"
#include "gemm.h"

namespace muon {

namespace {

constexpr int kMaxItems = 64;
constexpr int kRowsPerUnit = 4;     // rows a warp has in flight
constexpr int kSegCols = 256;       // columns a warp covers

struct Item {
    const signed char* q;
    const unsigned char* e;
    const void* x;
    long long ldq, lde, ldx, unit_begin;
    int rows, cols, segs, vec;
};

struct ItemParams {
    Item it[kMaxItems];
    int n;
    long long units;
    int* d_status;
};

template <int DT, bool ENCODE>
__global__ void __launch_bounds__(256) act8_kernel(const __grid_constant__ ItemParams p) {
    const int lane = threadIdx.x & 31;
    const long long nwarps = (long long)gridDim.x * (blockDim.x >> 5);
    int ei = 0;
    bool bad = false;
    for (long long u = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); u < p.units; u += nwarps) {
        while (ei + 1 < p.n && u >= p.it[ei + 1].unit_begin) ++ei;
        const Item& I = p.it[ei];
        const long long local = u - I.unit_begin;
        const long long rg = local / I.segs;
        const int col = (int)(local - rg * I.segs) * kSegCols + lane * 8;
        const int row0 = (int)(rg * kRowsPerUnit);
        const int nvalid = min(8, max(0, I.cols - col));
        const bool vec = I.vec && nvalid == 8;
        if (ENCODE) {
            float x[kRowsPerUnit][8];
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r)
                load8_dt(I.x, (row0 + r) * I.ldx + col, DT, vec && row0 + r < I.rows,
                         row0 + r < I.rows ? nvalid : 0, x[r]);
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r) {
                const long long row = row0 + r;
                bad |= !act8_encode8(x[r], col, row < I.rows ? nvalid : 0, const_cast<signed char*>(I.q) + row * I.ldq,
                                     const_cast<unsigned char*>(I.e) + row * I.lde, lane);
            }
        } else {
            uint2 w[kRowsPerUnit];
            int b[kRowsPerUnit];
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r) {
                const long long row = row0 + r;
                const int nv = row < I.rows ? nvalid : 0;
                w[r] = act8_load8(I.q + row * I.ldq, col, nv);
                b[r] = nv > 0 ? I.e[row * I.lde + col / kActBlock] : 0;
            }
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r) {
                float v[8];
                act8_decode8(w[r], b[r], v);
                store8_dt(const_cast<void*>(I.x), (row0 + r) * I.ldx + col, DT, vec && row0 + r < I.rows,
                          row0 + r < I.rows ? nvalid : 0, v);
            }
        }
    }
    if (ENCODE && __syncthreads_or(bad) && threadIdx.x == 0 && p.d_status) atomicOr(p.d_status, MUON_FLAG_NONFINITE);
}

template <bool ENCODE>
muon_status run_items(const muon_act8_item* items, int n, int dt, int* d_status, cudaStream_t stream) {
    if (!items || n < 1 || (dt != DT_BF16 && dt != DT_FP16 && dt != DT_FP32)) return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const muon_act8_item& q = items[i];
        if (!act8_valid(q.c) || q.ldx < q.c.cols || (q.c.rows > 0 && !q.x)) return MUON_ERR_INVALID_ARG;
    }
    const muon_status st = check_device();
    if (st != MUON_OK) return st;
    static ItemParams prm;             // large: kept off the stack, filled and consumed per launch
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    for (int b = 0; b < n; b += kMaxItems) {
        memset(&prm, 0, sizeof(prm));
        double bytes = 0.0;
        for (int i = b; i < std::min(n, b + kMaxItems); ++i) {
            const muon_act8_item& q = items[i];
            if (q.c.rows == 0) continue;
            Item& I = prm.it[prm.n++];
            I.q = q.c.q; I.e = q.c.e; I.x = q.x;
            I.ldq = q.c.ldq; I.lde = q.c.lde; I.ldx = q.ldx;
            I.rows = q.c.rows; I.cols = q.c.cols;
            I.segs = (q.c.cols + kSegCols - 1) / kSegCols;
            I.vec = rows_aligned(q.x, q.ldx, dt_size(dt));
            I.unit_begin = prm.units;
            prm.units += (long long)I.segs * ((q.c.rows + kRowsPerUnit - 1) / kRowsPerUnit);
            bytes += (double)q.c.rows * (q.c.cols * (dt_size(dt) + 1.0) + act8_blocks(q.c.cols));
        }
        if (prm.n == 0) continue;
        prm.d_status = d_status;
        int dev = 0, nsm = 148;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        const int grid = (int)std::min<long long>((prm.units + 7) / 8, (long long)nsm * 8);
        trace_begin(MUON_KERNEL_ACT8, bytes, stream);
        if (dt == DT_BF16) act8_kernel<DT_BF16, ENCODE><<<grid, 256, 0, stream>>>(prm);
        else if (dt == DT_FP16) act8_kernel<DT_FP16, ENCODE><<<grid, 256, 0, stream>>>(prm);
        else act8_kernel<DT_FP32, ENCODE><<<grid, 256, 0, stream>>>(prm);
        trace_end(stream);
        if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
    }
    return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status act8_encode_batched(const muon_act8_item* items, int n, muon_dtype x_dtype, int* d_status,
                                muon_stream_t stream) {
    return run_items<true>(items, n, x_dtype, d_status, reinterpret_cast<cudaStream_t>(stream));
}

muon_status act8_decode_batched(const muon_act8_item* items, int n, muon_dtype x_dtype, muon_stream_t stream) {
    return run_items<false>(items, n, x_dtype, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
