// act8.cu -- writing and reading 8-bit activation checkpoints (act8.cuh has the
// format).
//
// Both passes are bound by HBM: 2 + 1 + 1/32 bytes per element for 16-bit
// data (8192 x 14336 bfloat16: encode 59 us, 6.0 TB/s, decode 63 us, 5.65 TB/s).  A warp takes a segment of up to 256 columns of eight rows (of more rows where
// they are shorter), eight columns per lane (16-byte accesses of 16-bit data, 8-byte
// accesses of codes), every load issued before any use; a block's four lanes find its
// exponent with two shuffles.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "act8.cuh"
#include "gemm.h"

namespace muon {

namespace {

constexpr int kMaxItems = 64;
constexpr int kRowsPerUnit = 8;     // rows a warp has in flight

struct Item {
    const signed char* q;
    const unsigned char* e;
    const void* x;
    long long ldq, lde, ldx;
    uint32_t unit_begin, segs;
    int rows, cols, vec, lanes_log;
};

struct ItemParams {
    Item it[kMaxItems];
    int n;
    uint32_t units;
    int* d_status;
};

// Rows of x that cannot be taken in whole 16-byte pieces.  Encoding, a lane loads its
// eight columns one by one (the codes' rows are aligned all the same); decoding, it
// takes one column of every block, so that the warp's stores are whole runs of 32
// (eight single stores per lane, 16 bytes apart, took 2.1 times as long at 16384 x 1003).
template <int DT>
__device__ __forceinline__ bool encode_row(const char* x, signed char* q, unsigned char* e, int col, int cols, int lane) {
    const int nv = min(8, max(0, cols - col));
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < nv ? ld_elem(x, col + i, DT) : 0.f;
    return act8_encode8(v, col, nv, q, e, lane);
}

template <int DT>
__device__ __forceinline__ void decode_row(char* x, const signed char* q, const unsigned char* e, int col, int cols) {
    int code[8], byte[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = col + i * 32;
        code[i] = c < cols ? q[c] : 0;
        byte[i] = c < cols ? e[c / kActBlock] : 0;
    }
    float v[8];
    bool high = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = (float)code[i] * act8_step(byte[i]);
        high |= byte[i] >= kActFp16Top;
    }
    if (DT == DT_FP16 && __any_sync(0xFFFFFFFFu, high))
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act8_fp16(v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i * 32 < cols) st_elem(x, col + i * 32, DT, v[i]);
}

template <int DT, bool ENCODE>
__global__ void __launch_bounds__(256, DT != DT_FP32 ? 4 : ENCODE ? 2 : 3) act8_kernel(const __grid_constant__ ItemParams p) {
    constexpr int esz = DT == DT_FP32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const uint32_t nwarps = gridDim.x * (blockDim.x >> 5);
    int ei = 0;
    bool bad = false;
    for (uint32_t u = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); u < p.units; u += nwarps) {
        while (ei + 1 < p.n && u >= p.it[ei + 1].unit_begin) ++ei;
        const Item& I = p.it[ei];
        const uint32_t local = u - I.unit_begin, rg = local / I.segs, seg = local - rg * I.segs;
        char* x = static_cast<char*>(const_cast<void*>(I.x));
        signed char* q = const_cast<signed char*>(I.q);
        unsigned char* e = const_cast<unsigned char*>(I.e);
        if (!I.vec) {
#pragma unroll 4
            for (int r = 0; r < kRowsPerUnit; ++r) {
                const long long row = (long long)rg * kRowsPerUnit + r;
                if (row >= I.rows) break;
                if (ENCODE)
                    bad |= !encode_row<DT>(x + row * I.ldx * esz, q + row * I.ldq, e + row * I.lde, (int)seg * 256 + lane * 8,
                                           I.cols, lane);
                else
                    decode_row<DT>(x + row * I.ldx * esz, q + row * I.ldq, e + row * I.lde, (int)seg * 256 + lane, I.cols);
            }
            continue;
        }
        // 2^lanes_log lanes per row; kRowsPerUnit rows per lane, 32 >> lanes_log apart
        const int apart = 32 >> I.lanes_log, col = (int)((seg << I.lanes_log) + (lane & ((1 << I.lanes_log) - 1))) * 8;
        const long long row0 = (long long)rg * (kRowsPerUnit * apart) + (lane >> I.lanes_log);
        const int rows = (int)min((long long)kRowsPerUnit, (I.rows - row0 + apart - 1) / apart);     // of this lane; may be 0
        const bool in = col < I.cols;                          // eight columns or none
        x += (row0 * I.ldx + col) * esz;
        q += row0 * I.ldq + col;
        e += row0 * I.lde + col / kActBlock;
        const long long xstep = apart * I.ldx * esz, qstep = apart * I.ldq, estep = apart * I.lde;
        if (ENCODE) {
            Raw8<DT> raw[kRowsPerUnit];
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r, x += xstep) raw[r].load(x, in && r < rows);
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r, q += qstep, e += estep) {
                float v[8];
                uint2 w;
                raw[r].get(v);
                const int byte = act8_quantise8(v, w);
                if (in && r < rows) {
                    *reinterpret_cast<uint2*>(q) = w;
                    if ((lane & 3) == 0) *e = (unsigned char)byte;
                }
                bad |= byte == kActBad;
            }
        } else {
            // fp32: two runs of four columns per lane, so that a warp's 16-byte stores leave no gaps
            constexpr int kRuns = DT == DT_FP32 ? 2 : 1;
            const int sub = lane & ((1 << I.lanes_log) - 1);
            uint2 w[kRowsPerUnit];
            int b[kRowsPerUnit][kRuns];
            int c0 = 0, c1 = 0;                                // columns of the runs, from `col` on
            if (DT == DT_FP32) {
                c0 = -4 * sub;
                c1 = c0 + (4 << I.lanes_log);
            }
            const bool in0 = col + c0 < I.cols, in1 = col + c1 < I.cols;
            const int e0 = (col + c0) / kActBlock - col / kActBlock, e1 = (col + c1) / kActBlock - col / kActBlock;
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r, q += qstep, e += estep) {
                const bool ok = in0 && r < rows, ok1 = in1 && r < rows;
                if constexpr (DT == DT_FP32) {
                    w[r].x = ok ? *reinterpret_cast<const uint32_t*>(q + c0) : 0u;
                    w[r].y = ok1 ? *reinterpret_cast<const uint32_t*>(q + c1) : 0u;
                    b[r][1] = ok1 ? e[e1] : 0;
                } else {
                    w[r] = ok ? *reinterpret_cast<const uint2*>(q) : make_uint2(0u, 0u);
                }
                b[r][0] = ok ? e[e0] : 0;
            }
            // fp16: whether one of the warp's blocks may hold 65536 (act8_fp16), asked once: 16384 x 4096 38 us as without
            // the question, 43 us with it in every row
            bool high = false;
            if constexpr (DT == DT_FP16) {
#pragma unroll
                for (int r = 0; r < kRowsPerUnit; ++r) high |= b[r][0] >= kActFp16Top;
                high = __any_sync(0xFFFFFFFFu, high);
            }
            if (DT == DT_FP16 && high) {
#pragma unroll 1
                for (int r = 0; r < kRowsPerUnit; ++r) {
                    // again from memory: a loop that is not unrolled cannot index registers
                    if (!(in0 && r < rows)) continue;
                    float v[8];
                    const long long back = (long long)(kRowsPerUnit - r);
                    act8_decode8(*reinterpret_cast<const uint2*>(q - back * qstep), e[-back * estep], v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = act8_fp16(v[i]);
                    Raw8<DT> o;
                    o.set(v);
                    o.store(x + r * xstep, true);
                }
                continue;
            }
#pragma unroll
            for (int r = 0; r < kRowsPerUnit; ++r, x += xstep) {
                float v[8];
                if constexpr (DT == DT_FP32) {
                    float u[8];
                    act8_decode8(w[r], b[r][0], v);
                    act8_decode8(w[r], b[r][1], u);
                    if (in0 && r < rows) reinterpret_cast<float4*>(x + c0 * esz)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    if (in1 && r < rows) reinterpret_cast<float4*>(x + c1 * esz)[0] = make_float4(u[4], u[5], u[6], u[7]);
                } else {
                    Raw8<DT> o;
                    act8_decode8(w[r], b[r][0], v);
                    o.set(v);
                    o.store(x, in && r < rows);
                }
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
            I.vec = rows_aligned(q.x, q.ldx, dt_size(dt)) && q.c.cols % 8 == 0;
            // lanes of a row: a warp over one row of 256 columns or more, over several shorter ones
            I.lanes_log = 5;
            while (I.vec && I.lanes_log > 2 && (8 << (I.lanes_log - 1)) >= q.c.cols) --I.lanes_log;
            I.segs = (uint32_t)((q.c.cols + (8 << I.lanes_log) - 1) / (8 << I.lanes_log));
            const int unit_rows = kRowsPerUnit * (32 >> I.lanes_log);
            I.unit_begin = prm.units;
            const unsigned long long u = prm.units + (unsigned long long)I.segs * (((unsigned long long)q.c.rows + unit_rows - 1) / unit_rows);
            if (u > 0x7FFFFFFFu) return MUON_ERR_UNSUPPORTED;      // over 2^41 elements
            prm.units = (uint32_t)u;
            bytes += (double)q.c.rows * (q.c.cols * (dt_size(dt) + 1.0) + act8_blocks(q.c.cols));
        }
        if (prm.n == 0) continue;
        prm.d_status = d_status;
        int dev = 0, nsm = 148;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        const int grid = (int)std::min<long long>((prm.units + 7) / 8, (long long)nsm * 16);
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
