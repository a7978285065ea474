// seam.cu -- the seam between two blocks: norm behind a block, gate, residual
// scale, residual sum and the norm ahead of the next block in one pass, and the
// gradients of all of it from 8-bit checkpoints of the normalised rows
// (formulas at muon_seam and muon_seam_grad in muon.h).
//
// Both passes are bound by HBM.  A row lives in the registers of one block (VPT chunks
// of 8 consecutive columns per thread), so that the two norms of a seam, the second of
// which depends on every element the first has made, cost one read of the inputs.  Sums
// over a row: warp shuffles, then one round through shared memory, in a fixed
// order.  Sums over tokens (backward): every block takes a run of consecutive rows, keeps
// its columns' sums in registers and writes them once; a second launch adds the runs in
// order.
//
// 16384 x 4096 bfloat16, two RMS norms: forward 125 us (5.4 TB/s), with a gate per token or shared by 2048 tokens
// 150 us; backward 184 us (3.7 TB/s), with a gate per token 212 us, where the registers that rows, vectors' sums and
// checkpoints take leave 16 warps per SM, too few to hide the row's chain of sums behind other rows; with a shared gate
// 240 us (the same warps, sums that spill).  Two layer norms 185 us (shared memory for four vectors leaves 16 warps
// per SM) and 283 us (225 registers: 8 warps per SM).  Checkpoint values formed again from their codes where
// they are used, instead of kept, spilled less and issued more: slower.
//
// Two forms of each pass.  Where every row can be read in 16-byte pieces, a block
// has exactly the warps its rows need, and each thread copies its own pieces of the next
// rows into shared memory (cp.async, no barrier: nobody else reads them) while it
// works on this one.  Rows of other alignments (ANY) are copied as 4-byte words by the warp that
// works on them and written as runs of elements.
#include <algorithm>
#include <cmath>

#include "act8.cuh"
#include "gemm.h"

namespace muon {

namespace {

template <typename T> struct DtOf;
template <> struct DtOf<__nv_bfloat16> { static constexpr int v = DT_BF16; };
template <> struct DtOf<__half> { static constexpr int v = DT_FP16; };
template <> struct DtOf<float> { static constexpr int v = DT_FP32; };

// Backward: the runs of rows.
constexpr int kPlanSms = 148;       // runs are planned for a whole B200, so a size query needs no device

enum Vec : int { V_POST_GAIN, V_POST_BIAS, V_PRE_GAIN, V_PRE_BIAS, V_COUNT };

// Rows cut into runs, one per block.  A run holds whole gate groups (direct: their
// sums are finished in the run), or lies inside one group of which `parts` runs
// share the rows.
struct RunPlan {
    long long runs;
    int run_rows;      // rows of a run
    int parts;         // runs per gate group (0: the runs hold whole groups)
};

// The number of runs is that of the blocks that 1024 threads per SM make.  Forms with bias or gate sums hold fewer
// (16384 x 768 with bias sums: 6 blocks of 3 warps per SM for 10 planned, so 1366 runs in 1.5 rounds).
RunPlan plan_runs(int rows, int cols, int gate_rows, bool gate_sums) {
    const int threads = (cols + 255) / 256 * 32, per_sm = std::max(1, std::min(16, 1024 / threads));
    RunPlan P;
    const long long want = (long long)kPlanSms * per_sm;
    P.run_rows = (int)std::max<long long>(1, (rows + want - 1) / want);
    P.parts = 0;
    P.runs = (rows + P.run_rows - 1) / P.run_rows;
    if (gate_sums) {
        const long long groups = ((long long)rows + gate_rows - 1) / gate_rows;
        if (gate_rows <= P.run_rows) {
            P.run_rows = P.run_rows / gate_rows * gate_rows;
            P.runs = (rows + P.run_rows - 1) / P.run_rows;
        } else {
            const int span = std::min(gate_rows, rows);
            P.parts = (span + P.run_rows - 1) / P.run_rows;
            P.run_rows = (span + P.parts - 1) / P.parts;
            P.runs = groups * P.parts;
        }
    }
    return P;
}

struct BwdParams {
    muon_seam_grad s;
    RunPlan plan;
    float inv_c;
    int w_dt, vec, wvec, gate_sums;
    int vecs_in_smem, vectors, units;
    float* part;           // [V_COUNT + 1][runs][cols]: sums of one run (the last: shared gate rows)
};

// ---------------------------------------------------------------------------
// Rows in 16-byte pieces
// ---------------------------------------------------------------------------

// Sums of N values over a block of nw warps; every thread gets them.  `red`: two areas
// of 2 x 32 floats in turn, so one barrier per call is enough; entries of warps that do
// not exist stay 0.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red, int& slot, int nw) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    if (nw == 1) return;
    float* s = red + slot * 64;
    slot ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k * 32 + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
    if (nw <= 8) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float4 a = *reinterpret_cast<const float4*>(s + k * 32);
            v[k] = (a.x + a.y) + (a.z + a.w);
            if (nw > 4) {
                const float4 b = *reinterpret_cast<const float4*>(s + k * 32 + 4);
                v[k] += (b.x + b.y) + (b.z + b.w);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float t = s[k * 32 + (threadIdx.x & 31)];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
            v[k] = t;
        }
    }
}

// Normalise the row in v (columns beyond the row, nv columns into a chunk, hold 0 and stay 0):
// returns the reciprocal deviation.  The variance is summed over v - m, so that it does not cancel where the
// mean is large against the deviation; the mean m itself is an fp32 sum, off by up to 42 2^-24 mean|v| (42
// roundings; typically two), and so is every n by that times r: 0.025 at most for fp32 rows whose mean is 1e4 deviations.
// (The left-over mean summed beside the squares and taken off, too: 16384 x 4096 185 -> 205 us, and 124 -> 135 us for RMS
// norms, whose loop outgrows the instruction cache with it; only for rows far from zero, behind a branch, 200 and 133 us.)
// A sum of squares beyond fp32's range is formed again at 2^-100.
template <int VPT>
__device__ __forceinline__ float normalise(float (&v)[VPT][8], const int (&nv)[VPT], int kind, float eps, float inv_c,
                                           float* red, int& slot, int nw) {
    if (kind == MUON_NORM_LAYER) {
        float m[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) m[0] = fmaf(v[j][i], inv_c, m[0]);
        block_sum<1>(m, red, slot, nw);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = i < nv[j] ? v[j][i] - m[0] : 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(v[j][i], v[j][i], s[0]);
    block_sum<1>(s, red, slot, nw);
    float r;
    if (s[0] == __uint_as_float(0x7F800000u)) {      // uniform over the block
        const float down = __uint_as_float((127u - 100u) << 23);
        s[0] = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] = fmaf(v[j][i] * down, v[j][i] * down, s[0]);
        block_sum<1>(s, red, slot, nw);
        r = rsqrtf(s[0] * inv_c) * down;
    } else {
        r = rsqrtf(fmaf(s[0], inv_c, eps));
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] *= r;
    return r;
}

// A gain or bias times a constant (NULL: the constant alone, or nothing) on a thread's
// chunks, in shared memory as fp32 (two planes of four columns of every chunk, so that a
// warp's 16-byte reads leave no gaps; columns beyond the row hold 0) or, for rows whose
// vectors do not fit, read from global memory each time.
struct Vectors {
    float* sm;              // NULL: global
    int chunks, dt;         // chunks of a vector in shared memory: those of all threads
    int cols, vec;          // vec: 16-byte accesses of whole chunks
    __device__ __forceinline__ void get(int slot, const void* g, float mul, int col, bool in, float (&v)[8]) const {
        if (sm) {
            const float4 a = *reinterpret_cast<const float4*>(sm + 2 * slot * chunks * 4 + col / 2);
            const float4 b = *reinterpret_cast<const float4*>(sm + (2 * slot + 1) * chunks * 4 + col / 2);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            load(g, mul, col, in, v);
        }
    }
    __device__ __forceinline__ void load(const void* g, float mul, int col, bool in, float (&v)[8]) const {
        if (g) {
            load8_dt(g, col, dt, in && vec, in ? min(8, cols - col) : 0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= mul;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = in ? mul : 0.f;      // beyond the row's end it meets zeros
        }
    }
    // fill one vector of `cols` columns (before a barrier)
    __device__ __forceinline__ void fill(int slot, const void* g, float mul) const {
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            float v[8];
            load(g, mul, c * 8, c * 8 < cols, v);
            *reinterpret_cast<float4*>(sm + 2 * slot * chunks * 4 + c * 4) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(sm + (2 * slot + 1) * chunks * 4 + c * 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
};

// One thread's 16-byte pieces of the next rows: stage d, unit u of the stage's units,
// chunk j.
template <int VPT>
struct Ring {
    uint8_t* base;          // this thread's first piece
    int stride, units;      // bytes between pieces (16 x threads); units of a stage
    __device__ __forceinline__ uint8_t* at(int d, int u, int j) const { return base + ((d * units + u) * VPT + j) * stride; }
};

// One 16-byte copy; an fp32 chunk is two of them, halves of one sector.
template <int NPC>
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    if (NPC == 2) cp_async16_l1(dst, src);
    else cp_async16(dst, src, 16);
}

// Eight elements of a thread's chunk from the ring (zeros for a thread without columns: it never copies, and
// its pieces were cleared).
template <int DT, int VPT>
__device__ __forceinline__ void ring_get(const Ring<VPT>& ring, int d, int u, int j, float (&v)[8]) {
    Raw8<DT> r;
#pragma unroll
    for (int n = 0; n < Raw8<DT>::N; ++n) r.w[n] = *reinterpret_cast<const uint4*>(ring.at(d, u + n, j));
    r.get(v);
}

// Rows of any alignment (ANY).  The 256 columns of a warp's chunk are copied by its lanes in
// turn as the aligned 4-byte words that hold them, and written back through shared memory as
// whole runs of elements; a warp exchanges its data only with itself.  A row of 16-bit
// elements that starts in the middle of a word (`shift`) is read two bytes on, and the word behind the
// warp's 512 bytes has a place of its own.
template <typename T, int VPT>
struct AnyRow {
    const Ring<VPT>& ring;
    uint32_t* extra;        // this warp's words behind its chunks: one per piece of the ring, `warps` apart
    int warps, lane;

    __device__ __forceinline__ uint32_t* behind(int d, int u, int j) const {
        return extra + ((d * ring.units + u) * VPT + j) * warps;
    }
    // columns seg .. seg + 255 of a row
    __device__ __forceinline__ void copy(int d, int u, int j, const T* row, int seg, int cols) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(row + seg);
        uint8_t* base = ring.at(d, u, j) - lane * 16;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = i * 32 + lane;
                if (seg + c < cols)
                    cp_async4(ring.at(d, u + ((c >> 2) & 1), j) - lane * 16 + (c >> 3) * 16 + (c & 3) * 4,
                              reinterpret_cast<const void*>(a + 4 * c), 4u);
            }
        } else {
            const int bytes = (int)(a & 2) + 2 * min(256, cols - seg);      // from the first word on
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int w = (i * 32 + lane) * 4;
                if (w < bytes) cp_async4(base + w, reinterpret_cast<const void*>((a & ~uintptr_t(3)) + w), 4u);
            }
            if (lane == 0 && bytes > 512) cp_async4(behind(d, u, j), reinterpret_cast<const void*>((a & ~uintptr_t(3)) + 512), 4u);
        }
    }
    // this lane's eight columns, nv of them in the row
    __device__ __forceinline__ void get(int d, int u, int j, const T* row, int nv, float (&v)[8]) const {
        constexpr int DT = DtOf<T>::v;
        Raw8<DT> r;
#pragma unroll
        for (int n = 0; n < Raw8<DT>::N; ++n) r.w[n] = *reinterpret_cast<const uint4*>(ring.at(d, u + n, j));
        if constexpr (sizeof(T) == 2) {
            if (reinterpret_cast<uintptr_t>(row) & 2) {
                const uint32_t next = lane < 31 ? *reinterpret_cast<const uint32_t*>(ring.at(d, u, j) + 16) : *behind(d, u, j);
                uint4& w = r.w[0];
                w = make_uint4(__byte_perm(w.x, w.y, 0x5432), __byte_perm(w.y, w.z, 0x5432), __byte_perm(w.z, w.w, 0x5432),
                               __byte_perm(w.w, next, 0x5432));
            }
        }
        r.get(v);
        if (nv < 8)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < nv ? v[i] : 0.f;
    }
    // write the columns through the places of the first stream's pieces, which have been read
    template <typename U>
    __device__ __forceinline__ void put(int d, int j, U* row, int seg, int cols, const float (&v)[8]) const {
        Raw8<DtOf<U>::v> o;
        o.set(v);
        __syncwarp();
#pragma unroll
        for (int n = 0; n < o.N; ++n) *reinterpret_cast<uint4*>(ring.at(d, n, j)) = o.w[n];
        __syncwarp();
        if (seg < cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = i * 32 + lane;
                const uint8_t* p = sizeof(U) == 4 ? ring.at(d, (c >> 2) & 1, j) - lane * 16 + (c >> 3) * 16 + (c & 3) * 4
                                                  : ring.at(d, 0, j) - lane * 16 + c * 2;
                if (seg + c < cols) row[seg + c] = *reinterpret_cast<const U*>(p);
            }
        }
        __syncwarp();
    }
};

struct FwdParams {
    muon_seam s;
    float inv_c;
    int w_dt, vec, wvec;
    int sectors;           // fp32 rows that are written allow 32-byte accesses
    int vecs_in_smem, vectors, units;
    int* d_status;
};

enum FwdVec : int { F_POST_GAIN, F_PRE_GAIN, F_POST_BIAS, F_PRE_BIAS, F_VECS };   // the biases only where there is one

constexpr int kRedBytes = 512;      // block_sum's areas

// D rows are in flight or at work; MINB blocks of MAXT threads per SM bound the registers.  WARP: every
// warp of the block has rows of its own (rows of up to 1024 columns: no barriers, and the block's
// warps share its vectors).
template <typename T, int VPT, int MAXT, int D, int MINB, bool WARP, bool ANY>
__global__ void __launch_bounds__(MAXT, MINB) seam_fwd_kernel(const __grid_constant__ FwdParams p) {
    constexpr int DT = DtOf<T>::v;
    constexpr int NPC = sizeof(T) == 4 ? 2 : 1, kF = NPC, kGate = 2 * NPC;        // units of a stage (x first)
    extern __shared__ __align__(16) uint8_t smem[];
    const muon_seam& S = p.s;
    float* red = reinterpret_cast<float*>(smem);
    const int lane = threadIdx.x & 31, threads = WARP ? 32 : blockDim.x, nw = threads >> 5;      // of a row
    const int tr = WARP ? lane : (int)threadIdx.x;
    const bool has_f = S.f != nullptr, has_gate = S.gate != nullptr, has_pb = S.post_bias != nullptr;
    const bool has_yb = S.pre_bias != nullptr, unit_skip = S.skip == 1.f;
    const int post = S.post, pre = S.pre;
    for (int i = threadIdx.x; i < kRedBytes / 4; i += blockDim.x) red[i] = 0.f;
    // scale rides on the post-norm's vectors
    const Vectors V{p.vecs_in_smem ? reinterpret_cast<float*>(smem + kRedBytes) : nullptr, threads * VPT, p.w_dt, S.cols, !ANY};
    if (V.sm) {
        V.fill(F_POST_GAIN, S.post_gain, S.scale);
        V.fill(F_PRE_GAIN, S.pre_gain, 1.f);
        if (has_pb) V.fill(F_POST_BIAS, S.post_bias, S.scale);
        if (has_yb) V.fill(F_PRE_BIAS, S.pre_bias, 1.f);
    }
    const Ring<VPT> ring{smem + kRedBytes + (V.sm ? p.vectors * 32 * V.chunks : 0) + threadIdx.x * 16, (int)blockDim.x * 16, p.units};
    int col[VPT], nv[VPT];
    bool in[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        col[j] = (j * threads + tr) * 8;
        in[j] = col[j] < S.cols;
        nv[j] = max(0, min(8, S.cols - col[j]));
        if (!in[j])
            for (int u = 0; u < D * p.units; ++u) *reinterpret_cast<uint4*>(ring.at(0, u, j)) = make_uint4(0u, 0u, 0u, 0u);
    }
    uint8_t* after = smem + kRedBytes + (V.sm ? p.vectors * 32 * V.chunks : 0) + D * p.units * VPT * blockDim.x * 16;
    const AnyRow<T, VPT> any{ring, reinterpret_cast<uint32_t*>(after) + (threadIdx.x >> 5), (int)blockDim.x >> 5, lane};
    const int seg0 = (tr - lane) * 8;                      // the warp's first column of a chunk
    __syncthreads();
    const long long worker = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const long long workers = WARP ? (long long)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int r0 = (int)(S.rows * worker / workers), r1 = (int)(S.rows * (worker + 1) / workers);
    // this thread's first chunk of the next row to copy, and of the row at work
    const int t8 = ANY ? 0 : tr * 8;
    const T* x = static_cast<const T*>(S.x) + r0 * S.ldx + t8;
    const T* f = static_cast<const T*>(S.f) + r0 * S.ldf + t8;
    int grow = has_gate ? r0 / S.gate_rows : 0, gleft = has_gate ? S.gate_rows - r0 % S.gate_rows : 0;
    const T* gate = static_cast<const T*>(S.gate) + grow * S.ldgate + t8;
    T* out = static_cast<T*>(S.out) + r0 * S.ldout + t8;
    T* y = static_cast<T*>(S.y) + r0 * S.ldy + t8;
    signed char *pq = S.post_c.q + r0 * S.post_c.ldq + tr * 8, *yq = S.pre_c.q + r0 * S.pre_c.ldq + tr * 8;
    unsigned char *pe = S.post_c.e + r0 * S.post_c.lde, *ye = S.pre_c.e + r0 * S.pre_c.lde;
    const bool keep_f = S.post_c.q != nullptr, keep_y = S.pre_c.q != nullptr;
    auto copy = [&](int row, int d) {
        if (row < r1) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if constexpr (ANY) {
                    const int seg = seg0 + j * threads * 8;
                    if (seg >= S.cols) continue;
                    any.copy(d, 0, j, x, seg, S.cols);
                    if (has_f) any.copy(d, kF, j, f, seg, S.cols);
                    if (has_gate) any.copy(d, kGate, j, gate, seg, S.cols);
                    continue;
                }
                if (!in[j]) continue;
#pragma unroll
                for (int n = 0; n < NPC; ++n) {
                    const int c = j * threads * 8 + n * 4;
                    copy16<NPC>(ring.at(d, n, j), x + c);
                    if (has_f) copy16<NPC>(ring.at(d, kF + n, j), f + c);
                    if (has_gate) copy16<NPC>(ring.at(d, kGate + n, j), gate + c);
                }
            }
            x += S.ldx;
            f += S.ldf;
            if (has_gate && --gleft == 0) {
                gate += S.ldgate;
                gleft = S.gate_rows;
            }
        }
        cp_async_commit();
    };
    int slot = 0, d = 0;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < D - 1; ++k) copy(r0 + k, k);
    for (int row = r0; row < r1; ++row) {
        copy(row + D - 1, d == 0 ? D - 1 : d - 1);
        cp_async_wait<D - 1>();
        if (ANY) __syncwarp();                              // the other lanes' copies too
        float v[VPT][8];
        if (has_f) {
            float u[VPT][8];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if constexpr (ANY) any.get(d, kF, j, static_cast<const T*>(S.f) + row * S.ldf, nv[j], u[j]);
                else ring_get<DT, VPT>(ring, d, kF, j, u[j]);
            }
            if (post != MUON_NORM_NONE) {
                const float r = normalise<VPT>(u, nv, post, S.eps, p.inv_c, red, slot, nw);
                if (S.post_rstd && tr == 0) S.post_rstd[row] = r;
            }
            if (keep_f) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    uint2 w;
                    const int byte = act8_quantise8(u[j], w);
                    bad |= byte == kActBad;
                    if (ANY && nv[j] < 8) {
                        for (int i = 0; i < nv[j]; ++i) pq[j * threads * 8 + i] = (signed char)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
                        if ((lane & 3) == 0 && in[j]) pe[col[j] / kActBlock] = (unsigned char)byte;
                    } else if (in[j]) {
                        *reinterpret_cast<uint2*>(pq + j * threads * 8) = w;
                        if ((lane & 3) == 0) pe[col[j] / kActBlock] = (unsigned char)byte;
                    }
                }
                pq += S.post_c.ldq;
                pe += S.post_c.lde;
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float t[8];
                V.get(F_POST_GAIN, S.post_gain, S.scale, col[j], in[j], t);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[j][i] *= t[i];
                if (has_pb) {
                    V.get(F_POST_BIAS, S.post_bias, S.scale, col[j], in[j], t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[j][i] += t[i];
                }
                if constexpr (ANY) any.get(d, 0, j, static_cast<const T*>(S.x) + row * S.ldx, nv[j], v[j]);
                else ring_get<DT, VPT>(ring, d, 0, j, v[j]);
                if (!unit_skip)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] *= S.skip;
                if (has_gate) {
                    if constexpr (ANY)
                        any.get(d, kGate, j, static_cast<const T*>(S.gate) + (row / S.gate_rows) * S.ldgate, nv[j], t);
                    else
                        ring_get<DT, VPT>(ring, d, kGate, j, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = fmaf(u[j][i], t[i], v[j][i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] += u[j][i];
                }
                // fp32 in whole sectors: 16384 x 4096 203 us, 225 us with 16-byte stores (but rows per warp 52 us
                // against 50 at 16384 x 768, and the backward pass with a gate 486 us against 455)
                Raw8<DT> o;
                o.set(v[j]);
                if constexpr (ANY) any.put(d, j, out, seg0 + j * threads * 8, S.cols, v[j]);
                else o.store(out + j * threads * 8, in[j], !WARP && p.sectors);
                o.get(v[j]);                    // as it was stored
                if (ANY && nv[j] < 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = i < nv[j] ? v[j][i] : 0.f;
            }
            out += S.ldout;
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if constexpr (ANY) any.get(d, 0, j, static_cast<const T*>(S.x) + row * S.ldx, nv[j], v[j]);
                else ring_get<DT, VPT>(ring, d, 0, j, v[j]);
            }
        }
        if (pre != MUON_NORM_NONE) {
            const float r = normalise<VPT>(v, nv, pre, S.eps, p.inv_c, red, slot, nw);
            if (S.pre_rstd && tr == 0) S.pre_rstd[row] = r;
            if (keep_y) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    uint2 w;
                    const int byte = act8_quantise8(v[j], w);
                    bad |= byte == kActBad;
                    if (ANY && nv[j] < 8) {
                        for (int i = 0; i < nv[j]; ++i) yq[j * threads * 8 + i] = (signed char)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
                        if ((lane & 3) == 0 && in[j]) ye[col[j] / kActBlock] = (unsigned char)byte;
                    } else if (in[j]) {
                        *reinterpret_cast<uint2*>(yq + j * threads * 8) = w;
                        if ((lane & 3) == 0) ye[col[j] / kActBlock] = (unsigned char)byte;
                    }
                }
                yq += S.pre_c.ldq;
                ye += S.pre_c.lde;
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float t[8];
                V.get(F_PRE_GAIN, S.pre_gain, 1.f, col[j], in[j], t);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= t[i];
                if (has_yb) {
                    V.get(F_PRE_BIAS, S.pre_bias, 1.f, col[j], in[j], t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] += t[i];
                }
                Raw8<DT> o;
                o.set(v[j]);
                if constexpr (ANY) any.put(d, j, y, seg0 + j * threads * 8, S.cols, v[j]);
                else o.store(y + j * threads * 8, in[j], !WARP && p.sectors);
            }
            y += S.ldy;
        }
        d = d + 1 == D ? 0 : d + 1;
        if (ANY) __syncwarp();                              // this row is read before its place is copied to again
    }
    cp_async_wait<0>();
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0 && p.d_status) atomicOr(p.d_status, MUON_FLAG_NONFINITE);
}

enum BwdVec : int { B_POST_GAIN, B_PRE_GAIN, B_POST_BIAS, B_VECS };

template <typename T, int VPT, int MAXT, int D, int MINB, bool BIAS, bool GSUM, bool ANY>
__global__ void __launch_bounds__(MAXT, MINB) seam_bwd_kernel(const __grid_constant__ BwdParams p) {
    constexpr int DT = DtOf<T>::v;
    constexpr int NPC = sizeof(T) == 4 ? 2 : 1;
    constexpr int kDout = NPC, kCodes = 2 * NPC, kGate = 2 * NPC + 1;       // units of a stage (dy first)
    extern __shared__ __align__(16) uint8_t smem[];
    const muon_seam_grad& S = p.s;
    float* red = reinterpret_cast<float*>(smem);
    const int threads = blockDim.x, nw = threads >> 5;
    const bool has_pre = S.pre != MUON_NORM_NONE, has_post = S.post != MUON_NORM_NONE, has_f = S.df != nullptr;
    const bool has_dout = S.dout != nullptr, has_gate = S.gate != nullptr, post_c = S.post_c.q != nullptr;
    const bool has_pb = S.post_bias != nullptr, dgate = S.dgate != nullptr, gate_sums = GSUM && p.gate_sums;
    for (int i = threadIdx.x; i < kRedBytes / 4; i += threads) red[i] = 0.f;
    // scale rides on the post-norm's vectors
    const Vectors V{p.vecs_in_smem ? reinterpret_cast<float*>(smem + kRedBytes) : nullptr, threads * VPT, p.w_dt, S.cols, !ANY};
    if (V.sm) {
        V.fill(B_POST_GAIN, S.post_gain, S.scale);
        V.fill(B_PRE_GAIN, S.pre_gain, 1.f);
        if (has_pb) V.fill(B_POST_BIAS, S.post_bias, S.scale);
    }
    const Ring<VPT> ring{smem + kRedBytes + (V.sm ? p.vectors * 32 * V.chunks : 0) + threadIdx.x * 16, threads * 16, p.units};
    int col[VPT], ecol[VPT], nv[VPT];
    bool in[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        col[j] = (j * threads + (int)threadIdx.x) * 8;
        in[j] = col[j] < S.cols;
        nv[j] = max(0, min(8, S.cols - col[j]));
        ecol[j] = (in[j] ? col[j] : 0) / kActBlock;
        if (!in[j])
            for (int u = 0; u < D * p.units; ++u) *reinterpret_cast<uint4*>(ring.at(0, u, j)) = make_uint4(0u, 0u, 0u, 0u);
    }
    const int lane = threadIdx.x & 31;
    uint8_t* after = smem + kRedBytes + (V.sm ? p.vectors * 32 * V.chunks : 0) + D * p.units * VPT * threads * 16;
    const AnyRow<T, VPT> any{ring, reinterpret_cast<uint32_t*>(after) + (threadIdx.x >> 5), nw, lane};
    const int seg0 = ((int)threadIdx.x - lane) * 8;        // the warp's first column of a chunk
    __syncthreads();
    int r0, r1;
    if (p.plan.parts == 0) {
        r0 = (int)min((long long)S.rows, (long long)blockIdx.x * p.plan.run_rows);
        r1 = (int)min((long long)S.rows, (long long)r0 + p.plan.run_rows);
    } else {
        const long long g = blockIdx.x / p.plan.parts, end = min((long long)S.rows, (g + 1) * S.gate_rows);
        r0 = (int)min(end, g * S.gate_rows + (long long)(blockIdx.x % p.plan.parts) * p.plan.run_rows);
        r1 = (int)min(end, (long long)r0 + p.plan.run_rows);
    }
    const int gr = has_gate ? S.gate_rows : 1;
    int gleft = has_gate ? gr - r0 % gr : 0, cleft = gleft;                 // rows left of the gate row: of the next copy, at work
    // this thread's first chunk of the next row to copy, and of the row at work
    const int t8 = ANY ? 0 : threadIdx.x * 8;
    const T* dy = static_cast<const T*>(S.dy) + r0 * S.lddy + t8;
    const T* dout = static_cast<const T*>(S.dout) + r0 * S.lddout + t8;
    const T* gate = static_cast<const T*>(S.gate) + (r0 / gr) * S.ldgate + t8;
    const signed char* yq = S.pre_c.q + r0 * S.pre_c.ldq + threadIdx.x * 8;
    const signed char* pq = S.post_c.q + r0 * S.post_c.ldq + threadIdx.x * 8;
    T* dx = static_cast<T*>(S.dx) + r0 * S.lddx + t8;
    T* df = static_cast<T*>(S.df) + r0 * S.lddf + t8;
    T* dg = static_cast<T*>(S.dgate) + (r0 / gr) * S.lddgate + t8;
    auto copy = [&](int row, int d) {
        if (row < r1) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int cj = j * threads * 8;
                if constexpr (ANY) {
                    if (seg0 + cj < S.cols) {
                        if (has_pre) any.copy(d, 0, j, dy, seg0 + cj, S.cols);
                        if (has_dout) any.copy(d, kDout, j, dout, seg0 + cj, S.cols);
                        if (has_gate) any.copy(d, kGate, j, gate, seg0 + cj, S.cols);
                    }
                }
                if (!in[j]) continue;
                if constexpr (!ANY) {
#pragma unroll
                    for (int n = 0; n < NPC; ++n) {
                        if (has_pre) copy16<NPC>(ring.at(d, n, j), dy + cj + n * 4);
                        if (has_dout) copy16<NPC>(ring.at(d, kDout + n, j), dout + cj + n * 4);
                        if (has_gate) copy16<NPC>(ring.at(d, kGate + n, j), gate + cj + n * 4);
                    }
                }
                if (has_pre) cp_async8(ring.at(d, kCodes, j), yq + cj);
                if (post_c) cp_async8(ring.at(d, kCodes, j) + 8, pq + cj);
            }
            dy += S.lddy;
            dout += S.lddout;
            yq += S.pre_c.ldq;
            pq += S.post_c.ldq;
            if (has_gate && --gleft == 0) {
                gate += S.ldgate;
                gleft = gr;
            }
        }
        cp_async_commit();
    };
    // exponent bytes and deviations of the next row
    int ep[VPT], eq[VPT];
    float rp = 0.f, rq = 0.f;
    const unsigned char *ye = S.pre_c.e + r0 * S.pre_c.lde, *pe = S.post_c.e + r0 * S.post_c.lde;
    auto scalars = [&](int row) {
        if (row >= r1) return;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (has_pre) ep[j] = ye[ecol[j]];
            if (post_c) eq[j] = pe[ecol[j]];
        }
        ye += S.pre_c.lde;
        pe += S.post_c.lde;
        if (has_pre) rp = S.pre_rstd[row];
        if (has_post) rq = S.post_rstd[row];
    };
    // codes of a thread without columns are 0 under any finite scale; a bad block's byte must not reach them
    auto decode = [&](int d, int half, int j, int byte, float (&n)[8]) {
        act8_decode8(*reinterpret_cast<const uint2*>(ring.at(d, kCodes, j) + 8 * half), in[j] ? byte : 127, n);
        if (ANY && nv[j] < 8)
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = i < nv[j] ? n[i] : 0.f;
    };
    float a_pg[VPT][8] = {}, a_qg[VPT][8] = {};               // d_pre_gain, d_post_gain / scale
    float a_pb[BIAS ? VPT : 1][8] = {}, a_qb[BIAS ? VPT : 1][8] = {}, a_gt[GSUM ? VPT : 1][8] = {};
    int slot = 0, d = 0;
    scalars(r0);
#pragma unroll
    for (int k = 0; k < D - 1; ++k) copy(r0 + k, k);
    for (int row = r0; row < r1; ++row) {
        copy(row + D - 1, d == 0 ? D - 1 : d - 1);
        cp_async_wait<D - 1>();
        if (ANY) __syncwarp();                                // the other lanes' copies too
        const float r_pre = rp, r_post = rq;
        int b_pre[VPT], b_post[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            b_pre[j] = ep[j];
            b_post[j] = eq[j];
        }
        scalars(row + 1);
        float x[VPT][8];                                      // d, the gradient of x'
        if (has_pre) {
            float n[VPT][8], sums[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float t[8];
                if constexpr (ANY) any.get(d, 0, j, static_cast<const T*>(S.dy) + row * S.lddy, nv[j], x[j]);
                else ring_get<DT, VPT>(ring, d, 0, j, x[j]);
                decode(d, 0, j, b_pre[j], n[j]);
                V.get(B_PRE_GAIN, S.pre_gain, 1.f, col[j], in[j], t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float gn = x[j][i] * n[j][i];
                    a_pg[j][i] += gn;
                    if constexpr (BIAS) a_pb[j][i] += x[j][i];
                    sums[0] = fmaf(gn, t[i], sums[0]);
                    x[j][i] *= t[i];
                }
                if (S.pre == MUON_NORM_LAYER)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sums[1] += x[j][i];
            }
            float s0 = 0.f, s1;
            if (S.pre == MUON_NORM_LAYER) {
                block_sum<2>(sums, red, slot, nw);
                s0 = sums[1] * p.inv_c * r_pre;
                s1 = sums[0];
            } else {
                float one[1] = {sums[0]};
                block_sum<1>(one, red, slot, nw);
                s1 = one[0];
            }
            s1 *= p.inv_c * r_pre;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float t[8];
                if (has_dout) {
                    if constexpr (ANY) any.get(d, kDout, j, static_cast<const T*>(S.dout) + row * S.lddout, nv[j], t);
                    else ring_get<DT, VPT>(ring, d, kDout, j, t);
                }
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = 0.f;
                // columns beyond the row (t, x and n are 0) stay out of the sums over it
                const float s0j = in[j] ? s0 : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = fmaf(r_pre, x[j][i], fmaf(-s1, n[j][i], t[i] - s0j));
                if (ANY && nv[j] < 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j][i] = i < nv[j] ? x[j][i] : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if constexpr (ANY) any.get(d, kDout, j, static_cast<const T*>(S.dout) + row * S.lddout, nv[j], x[j]);
                else ring_get<DT, VPT>(ring, d, kDout, j, x[j]);
            }
        }
        if (has_f) {
            float n[VPT][8], h[VPT][8], sums[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float t[8];
                if (post_c) decode(d, 1, j, b_post[j], n[j]);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) n[j][i] = 0.f;
                V.get(B_POST_GAIN, S.post_gain, S.scale, col[j], in[j], t);
                if (has_gate) {
                    float g[8];
                    if constexpr (ANY) any.get(d, kGate, j, static_cast<const T*>(S.gate) + (row / gr) * S.ldgate, nv[j], g);
                    else ring_get<DT, VPT>(ring, d, kGate, j, g);
                    if (dgate) {
                        float u[8];
                        if (has_pb) {
                            V.get(B_POST_BIAS, S.post_bias, S.scale, col[j], in[j], u);
#pragma unroll
                            for (int i = 0; i < 8; ++i) u[i] = fmaf(n[j][i], t[i], u[i]) * x[j][i];
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) u[i] = n[j][i] * t[i] * x[j][i];
                        }
                        if (!gate_sums) {
                            Raw8<DT> o;
                            o.set(u);
                            if constexpr (ANY) any.put(d, j, dg, seg0 + j * threads * 8, S.cols, u);
                            else o.store(dg + j * threads * 8, in[j]);
                        }
                        if constexpr (GSUM) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) a_gt[j][i] += u[i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] = x[j][i] * g[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] = x[j][i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float hn = h[j][i] * n[j][i];
                    a_qg[j][i] += hn;
                    if constexpr (BIAS) a_qb[j][i] += h[j][i];
                    sums[0] = fmaf(hn, t[i], sums[0]);
                    h[j][i] *= t[i];
                }
                if (S.post == MUON_NORM_LAYER)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sums[1] += h[j][i];
            }
            if (has_post) {
                float s0 = 0.f, s1;
                if (S.post == MUON_NORM_LAYER) {
                    block_sum<2>(sums, red, slot, nw);
                    s0 = sums[1] * p.inv_c * r_post;
                    s1 = sums[0];
                } else {
                    float one[1] = {sums[0]};
                    block_sum<1>(one, red, slot, nw);
                    s1 = one[0];
                }
                s1 *= p.inv_c * r_post;
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] = fmaf(r_post, h[j][i], fmaf(-s1, n[j][i], -s0));
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                Raw8<DT> o;
                o.set(h[j]);
                if constexpr (ANY) any.put(d, j, df, seg0 + j * threads * 8, S.cols, h[j]);
                else o.store(df + j * threads * 8, in[j]);
            }
            df += S.lddf;
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (S.skip != 1.f)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] *= S.skip;
            Raw8<DT> o;
            o.set(x[j]);
            if constexpr (ANY) any.put(d, j, dx, seg0 + j * threads * 8, S.cols, x[j]);
            else o.store(dx + j * threads * 8, in[j]);
        }
        dx += S.lddx;
        if (has_gate && (--cleft == 0 || row + 1 == S.rows)) {
            if constexpr (GSUM) {
                if (gate_sums && p.plan.parts == 0) {
#pragma unroll
                    for (int j = 0; j < VPT; ++j) {
                        Raw8<DT> o;
                        o.set(a_gt[j]);
                        if constexpr (ANY) any.put(d, j, dg, seg0 + j * threads * 8, S.cols, a_gt[j]);
                        else o.store(dg + j * threads * 8, in[j]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) a_gt[j][i] = 0.f;
                    }
                }
            }
            dg += S.lddgate;
            cleft = gr;
        }
        d = d + 1 == D ? 0 : d + 1;
        if (ANY) __syncwarp();                                // this row is read before its place is copied to again
    }
    cp_async_wait<0>();
    auto put = [&](int v, float (&a)[8], float mul, int j) {
        Raw8<DT_FP32> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= mul;
        o.set(a);
        float* row = p.part + ((long long)v * p.plan.runs + blockIdx.x) * S.cols;
        if constexpr (ANY) any.put(0, j, row, seg0 + j * threads * 8, S.cols, a);
        else o.store(row + col[j], in[j]);
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (S.d_pre_gain) put(V_PRE_GAIN, a_pg[j], 1.f, j);
        if (S.d_post_gain) put(V_POST_GAIN, a_qg[j], S.scale, j);
        if constexpr (BIAS) {
            if (S.d_pre_bias) put(V_PRE_BIAS, a_pb[j], 1.f, j);
            if (S.d_post_bias) put(V_POST_BIAS, a_qb[j], S.scale, j);
        }
        if constexpr (GSUM)
            if (gate_sums && p.plan.parts) put(V_COUNT, a_gt[j], 1.f, j);
    }
}

// Sums of the runs' parts: blockIdx.y < V_COUNT a vector gradient (over every
// run), above that one shared gate row (over its runs).  32 columns x 32 lanes of
// runs; a lane adds its runs in order, the lanes are added in order.
__global__ void __launch_bounds__(1024) seam_join_kernel(const __grid_constant__ BwdParams p, int dt) {
    __shared__ float sm[32][33];
    const muon_seam_grad& S = p.s;
    const int c = blockIdx.x * 32 + threadIdx.x;
    int v = blockIdx.y;
    void* dst;
    long long first = 0, count = p.plan.runs, at = c;
    int odt = p.w_dt;
    float beta = S.beta;
    if (v < V_COUNT) {
        dst = v == V_POST_GAIN ? S.d_post_gain : v == V_POST_BIAS ? S.d_post_bias
              : v == V_PRE_GAIN ? S.d_pre_gain : S.d_pre_bias;
    } else {
        const long long g = v - V_COUNT;
        v = V_COUNT;
        dst = S.dgate;
        first = g * p.plan.parts;
        count = p.plan.parts;
        at = g * S.lddgate + c;
        odt = dt;
        beta = 0.f;
    }
    if (!dst) return;
    float s = 0.f;
    if (c < S.cols) {
        const float* src = p.part + ((long long)v * p.plan.runs + first) * S.cols + c;
#pragma unroll 8
        for (long long r = threadIdx.y; r < count; r += 32) s += src[r * S.cols];
    }
    sm[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < S.cols) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += sm[k][threadIdx.x];
        if (beta != 0.f) t = fmaf(beta, ld_elem(dst, at, odt), t);
        st_elem(dst, at, odt, t);
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool dtype_ok(int d) { return d == DT_BF16 || d == DT_FP16 || d == DT_FP32; }
bool norm_ok(int k) { return k == MUON_NORM_NONE || k == MUON_NORM_RMS || k == MUON_NORM_LAYER; }

// a kept checkpoint covers the seam's rows and columns
bool kept_ok(const muon_act8& c, int rows, int cols) {
    if (!c.q) return true;
    return c.rows == rows && c.cols == cols && act8_valid(c);
}

muon_status check_seam(const muon_seam* s) {
    if (!s || s->rows < 0 || s->rows > kActMaxDim || s->cols < 1 || !norm_ok(s->post) || !norm_ok(s->pre))
        return MUON_ERR_INVALID_ARG;
    if (!(s->eps > 0.f) || !std::isfinite(s->eps) || !std::isfinite(s->skip) || !std::isfinite(s->scale))
        return MUON_ERR_INVALID_ARG;
    if (s->cols > MUON_SEAM_MAX_COLS) return MUON_ERR_UNSUPPORTED;
    if (s->rows == 0) return MUON_OK;                  // nothing is read or written, pointers may be NULL
    const long long c = s->cols;
    const bool f = s->f != nullptr, pre = s->pre != MUON_NORM_NONE;
    if (!s->x || s->ldx < c || (f && s->ldf < c)) return MUON_ERR_INVALID_ARG;
    if (!f && (s->post != MUON_NORM_NONE || s->skip != 1.f || s->gate || s->post_gain || s->post_bias || s->post_c.q ||
               s->post_rstd || s->out))
        return MUON_ERR_INVALID_ARG;
    if (f && (!s->out || s->ldout < c)) return MUON_ERR_INVALID_ARG;
    if (s->post == MUON_NORM_NONE && s->post_rstd) return MUON_ERR_INVALID_ARG;     // there is none to receive
    if (s->gate && (s->ldgate < c || s->gate_rows < 1)) return MUON_ERR_INVALID_ARG;
    if (!pre && (s->y || s->pre_gain || s->pre_bias || s->pre_c.q || s->pre_rstd)) return MUON_ERR_INVALID_ARG;
    if (pre && (!s->y || s->ldy < c)) return MUON_ERR_INVALID_ARG;
    if (!f && !pre) return MUON_ERR_INVALID_ARG;       // nothing to make
    return kept_ok(s->post_c, s->rows, s->cols) && kept_ok(s->pre_c, s->rows, s->cols) ? MUON_OK : MUON_ERR_INVALID_ARG;
}

muon_status check_grad(const muon_seam_grad* s) {
    if (!s || s->rows < 0 || s->rows > kActMaxDim || s->cols < 1 || !norm_ok(s->post) || !norm_ok(s->pre))
        return MUON_ERR_INVALID_ARG;
    if (!std::isfinite(s->skip) || !std::isfinite(s->scale) || !std::isfinite(s->beta)) return MUON_ERR_INVALID_ARG;
    if (s->cols > MUON_SEAM_MAX_COLS) return MUON_ERR_UNSUPPORTED;
    if (s->rows == 0) return MUON_OK;                  // only the vector gradients are written (beta times what they hold)
    const long long c = s->cols;
    const bool pre = s->pre != MUON_NORM_NONE, f = s->df != nullptr;
    if (pre && (!s->dy || !s->pre_c.q || !s->pre_rstd || s->lddy < c)) return MUON_ERR_INVALID_ARG;
    if (!pre && (s->dy || s->pre_gain || s->d_pre_gain || s->d_pre_bias)) return MUON_ERR_INVALID_ARG;
    if (s->dout && s->lddout < c) return MUON_ERR_INVALID_ARG;
    if (!s->dx || s->lddx < c || !(pre || s->dout)) return MUON_ERR_INVALID_ARG;
    if (!f && (s->post != MUON_NORM_NONE || s->skip != 1.f || s->gate || s->dgate || s->post_gain || s->post_bias ||
               s->d_post_gain || s->d_post_bias))
        return MUON_ERR_INVALID_ARG;
    if (f && (s->lddf < c || s->df == s->dx)) return MUON_ERR_INVALID_ARG;
    if (s->gate && (s->ldgate < c || s->gate_rows < 1)) return MUON_ERR_INVALID_ARG;
    if (s->dgate && (!s->gate || s->lddgate < c)) return MUON_ERR_INVALID_ARG;
    if (s->post != MUON_NORM_NONE && !s->post_rstd) return MUON_ERR_INVALID_ARG;
    if (!s->post_c.q && (s->post != MUON_NORM_NONE || s->dgate || s->d_post_gain)) return MUON_ERR_INVALID_ARG;
    return kept_ok(s->post_c, s->rows, s->cols) && kept_ok(s->pre_c, s->rows, s->cols) ? MUON_OK : MUON_ERR_INVALID_ARG;
}

bool gate_sums(const muon_seam_grad& s) { return s.rows > 0 && s.dgate && s.gate_rows > 1; }
bool any_vector(const muon_seam_grad& s) { return s.d_post_gain || s.d_post_bias || s.d_pre_gain || s.d_pre_bias; }

size_t part_bytes(const muon_seam_grad& s, const RunPlan& P) {
    if (!any_vector(s) && !(gate_sums(s) && P.parts)) return 0;
    return (size_t)(V_COUNT + 1) * P.runs * s.cols * sizeof(float);
}

int sm_count() {
    int dev = 0, nsm = kPlanSms;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    return nsm;
}

// One form of a kernel: chunks of 8 columns per thread, most threads, stages, blocks per SM that
// its registers are bounded for; warp: a row per warp, blocks of maxt threads.
struct Form {
    int vpt, maxt, stages, per_sm;
    bool warp;
    int row_threads(int cols) const { return warp ? 32 : (cols + 256 * vpt - 1) / (256 * vpt) * 32; }
    int threads(int cols) const { return warp ? maxt : row_threads(cols); }
    // blocks that the registers of an SM take
    int blocks(int cols) const { return std::min(32, per_sm * maxt / threads(cols)); }
};

// Launches a form: its shared memory, with the vectors as fp32 wherever they fit (read from
// global memory they cost more than the blocks per SM that their space may cost: 16384 x 4096
// with a gate forward 150 us with three blocks and global vectors); the blocks that are resident then are
// the grid, unless the runs of rows are given.  The kernel's limit on shared memory is the device's whatever this
// call needs: another thread's call of the same kernel may set it between this one's setting and launch.
template <typename K, typename P>
cudaError_t seam_launch(K kern, P& p, const Form& f, bool any, long long runs, cudaStream_t s) {
    const int t = f.threads(p.s.cols), most = f.blocks(p.s.cols), room = 227 * 1024;
    const int ring = kRedBytes + f.stages * p.units * f.vpt * t * 16, vecs = p.vectors * 32 * f.vpt * f.row_threads(p.s.cols);
    const int more = any ? t / 32 * 4 * f.stages * p.units * f.vpt : 0;     // AnyRow's words behind the pieces
    p.vecs_in_smem = ring + more + vecs + 1024 <= room;
    const int smem = ring + more + (p.vecs_in_smem ? vecs : 0);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
    if (e != cudaSuccess) return e;
    const long long resident = (long long)sm_count() * std::max(1, std::min(most, room / (smem + 1024)));
    const long long most_blocks = ((long long)p.s.rows + t / f.row_threads(p.s.cols) - 1) / (t / f.row_threads(p.s.cols));
    kern<<<(unsigned)(runs ? runs : std::min(most_blocks, resident)), t, smem, s>>>(p);
    return cudaGetLastError();
}

// Rows of up to 1024 columns one per warp: no barriers, and a block shares its vectors (16384 x 768,
// layer norm, 25 us; a block per row 35 us).  Longer rows two chunks per thread, as many warps as
// the row needs (with four, half the warps fit their registers).
template <typename T>
cudaError_t launch_fwd(FwdParams& p, bool any, cudaStream_t s) {
    const int c = p.s.cols, npc = sizeof(T) == 4 ? 2 : 1;
    p.units = npc * (p.s.gate ? 3 : p.s.f ? 2 : 1);
    p.vectors = p.s.post_bias || p.s.pre_bias ? F_VECS : F_POST_BIAS;
#define SEAM_FWD(VPT, MAXT, D, MINB, WARP, ANY) \
    return seam_launch(seam_fwd_kernel<T, VPT, MAXT, D, MINB, WARP, ANY>, p, Form{VPT, MAXT, D, MINB, WARP}, ANY, 0, s)
    if (any) {
        if (c <= 1024) SEAM_FWD(4, 128, 2, 3, true, true);
        if (c <= 4096) SEAM_FWD(2, 256, 2, 2, false, true);
        if (c <= 8192) SEAM_FWD(2, 512, 2, 1, false, true);
        SEAM_FWD(2, 1024, 1, 1, false, true);
    }
    if (c <= 256) SEAM_FWD(1, 256, 3, 4, true, false);
    if (c <= 512) SEAM_FWD(2, 256, 2, 3, true, false);
    if (c <= 768) SEAM_FWD(3, 256, 2, 3, true, false);
    if (c <= 1024) SEAM_FWD(4, 128, 2, 4, true, false);
    if (c <= 4096) SEAM_FWD(2, 256, 2, 3, false, false);
    if (c <= 8192) SEAM_FWD(2, 512, 2, 1, false, false);
    SEAM_FWD(2, 1024, 1, 1, false, false);
#undef SEAM_FWD
}

// The sums over tokens take 8 to 40 registers per chunk, so short rows have one chunk per thread and a block
// each, and the forms with bias or shared gate sums, which few seams have, are compiled apart
// (16384 x 4096: two RMS norms 184 us, two layer norms with bias sums 283 us).  Rows of more than 8192 columns have
// 64 registers per thread and spill in every form: 4096 x 16384 362 us, two layer norms 563 us.
template <typename T, bool BIAS, bool GSUM, bool ANY>
cudaError_t launch_bwd_form(BwdParams& p, cudaStream_t s) {
    const int c = p.s.cols, npc = sizeof(T) == 4 ? 2 : 1;
    p.units = 2 * npc + 1 + (p.s.gate ? npc : 0);
    p.vectors = p.s.post_bias ? B_VECS : B_POST_BIAS;
#define SEAM_BWD(VPT, MAXT, D, MINB)                                                                                    \
    return seam_launch(seam_bwd_kernel<T, VPT, MAXT, D, MINB, BIAS, GSUM, ANY>, p, Form{VPT, MAXT, D, MINB, false}, ANY, p.plan.runs, s)
    if (c <= 768) SEAM_BWD(1, 96, 3, BIAS || GSUM ? 6 : 8);
    if (c <= 4096) SEAM_BWD(2, 256, 2, BIAS ? 1 : 2);
    if (c <= 8192) SEAM_BWD(2, 512, 2, 1);
    SEAM_BWD(2, 1024, 1, 1);
#undef SEAM_BWD
}

template <typename T>
cudaError_t launch_bwd(BwdParams& p, bool any, cudaStream_t s) {
    const bool bias = p.s.d_post_bias || p.s.d_pre_bias;
    if (any) return bias || p.gate_sums ? launch_bwd_form<T, true, true, true>(p, s) : launch_bwd_form<T, false, false, true>(p, s);
    if (p.gate_sums) return bias ? launch_bwd_form<T, true, true, false>(p, s) : launch_bwd_form<T, false, true, false>(p, s);
    return bias ? launch_bwd_form<T, true, false, false>(p, s) : launch_bwd_form<T, false, false, false>(p, s);
}

bool rows_sectors(const void* p, long long ld, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 31) == 0 && (ld * esz) % 32 == 0;
}
bool vec_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status seam_forward(const muon_seam* seam, muon_dtype x_dtype, muon_dtype w_dtype, int* d_status,
                         muon_stream_t stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return MUON_ERR_INVALID_ARG;
    muon_status st = check_seam(seam);
    if (st != MUON_OK) return st;
    st = check_device();
    if (st != MUON_OK) return st;
    if (seam->rows == 0) return MUON_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    FwdParams p;
    p.s = *seam;
    p.inv_c = 1.f / (float)seam->cols;
    p.w_dt = w_dtype;
    p.d_status = d_status;
    const int esz = dt_size(x_dtype);
    const muon_seam& q = *seam;
    p.vec = rows_aligned(q.x, q.ldx, esz) && (!q.f || (rows_aligned(q.f, q.ldf, esz) && rows_aligned(q.out, q.ldout, esz))) &&
            (!q.gate || rows_aligned(q.gate, q.ldgate, esz)) && (!q.y || rows_aligned(q.y, q.ldy, esz));
    p.sectors = (!q.f || rows_sectors(q.out, q.ldout, esz)) && (!q.y || rows_sectors(q.y, q.ldy, esz));
    p.wvec = vec_ok(q.post_gain) && vec_ok(q.post_bias) && vec_ok(q.pre_gain) && vec_ok(q.pre_bias);
    const double el = (double)q.rows * q.cols;
    trace_begin(MUON_KERNEL_SEAM, el * (esz * (1 + (q.f ? 2 : 0) + (q.y ? 1 : 0) + (q.gate && q.gate_rows == 1 ? 1 : 0)) +
                                        33.0 / 32 * ((q.post_c.q ? 1 : 0) + (q.pre_c.q ? 1 : 0))), s);
    const bool any = !(p.vec && p.wvec && q.cols % 8 == 0);
    const cudaError_t e = x_dtype == MUON_BF16   ? launch_fwd<__nv_bfloat16>(p, any, s)
                          : x_dtype == MUON_FP16 ? launch_fwd<__half>(p, any, s) : launch_fwd<float>(p, any, s);
    trace_end(s);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

muon_status seam_backward_workspace_size(const muon_seam_grad* seam, size_t* bytes) {
    if (!bytes) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_grad(seam);
    if (st != MUON_OK) return st;
    *bytes = part_bytes(*seam, plan_runs(seam->rows, seam->cols, seam->gate_rows, gate_sums(*seam)));
    return MUON_OK;
}

muon_status seam_backward(const muon_seam_grad* seam, muon_dtype x_dtype, muon_dtype w_dtype, void* workspace,
                          size_t ws_bytes, int* d_status, muon_stream_t stream) {
    (void)d_status;
    if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return MUON_ERR_INVALID_ARG;
    muon_status st = check_grad(seam);
    if (st != MUON_OK) return st;
    BwdParams p;
    p.s = *seam;
    const muon_seam_grad& q = *seam;
    p.gate_sums = gate_sums(q);
    p.plan = plan_runs(q.rows, q.cols, q.gate_rows, p.gate_sums);
    const size_t need = part_bytes(q, p.plan);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || ws_bytes < need))
        return MUON_ERR_WORKSPACE;
    st = check_device();
    if (st != MUON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.part = static_cast<float*>(workspace);
    p.inv_c = 1.f / (float)q.cols;
    p.w_dt = w_dtype;
    const int esz = dt_size(x_dtype);
    p.vec = (!q.dy || rows_aligned(q.dy, q.lddy, esz)) && (!q.dout || rows_aligned(q.dout, q.lddout, esz)) &&
            rows_aligned(q.dx, q.lddx, esz) && (!q.df || rows_aligned(q.df, q.lddf, esz)) &&
            (!q.gate || rows_aligned(q.gate, q.ldgate, esz)) && (!q.dgate || rows_aligned(q.dgate, q.lddgate, esz));
    p.wvec = vec_ok(q.post_gain) && vec_ok(q.post_bias) && vec_ok(q.pre_gain);
    const bool tok = q.gate && q.gate_rows == 1;
    if (p.plan.runs > 0) {
        trace_begin(MUON_KERNEL_SEAM, (double)q.rows * q.cols *
                        (esz * (1.0 + (q.dy ? 1 : 0) + (q.dout ? 1 : 0) + (q.df ? 1 : 0) + (tok ? 1 : 0) + (tok && q.dgate ? 1 : 0)) +
                         33.0 / 32 * ((q.dy ? 1 : 0) + (q.post_c.q ? 1 : 0))), s);
        const bool any = !(p.vec && p.wvec && q.cols % 8 == 0);
        const cudaError_t e = x_dtype == MUON_BF16   ? launch_bwd<__nv_bfloat16>(p, any, s)
                              : x_dtype == MUON_FP16 ? launch_bwd<__half>(p, any, s) : launch_bwd<float>(p, any, s);
        trace_end(s);
        if (e != cudaSuccess) return MUON_ERR_CUDA;
    }
    const long long groups = p.gate_sums && p.plan.parts ? p.plan.runs / p.plan.parts : 0;
    if (any_vector(q) || groups) {
        const int xt = (q.cols + 31) / 32;
        trace_begin(MUON_KERNEL_SEAM, 4.0 * p.plan.runs * q.cols, s);
        seam_join_kernel<<<dim3(xt, (unsigned)(V_COUNT + groups)), dim3(32, 32), 0, s>>>(p, x_dtype);
        trace_end(s);
        if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
    }
    return MUON_OK;
}

}  // extern "C"
