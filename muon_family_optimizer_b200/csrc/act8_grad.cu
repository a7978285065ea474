// act8_grad.cu -- weight gradients of linear layers from 8-bit activation
// checkpoints: G = beta G + (dY^T X^) diag(gain) + dy_sum shift^T.
//
// The sum runs over tokens, the rows of both operands, so both are read
// MN-major: A = dY^T (M = out) and B = X^ (N = cols), K = tokens.  X^ = q 2^e is
// exact in bfloat16, so the tensor cores take it as a 16-bit operand
// (kind::f16, fp32 accumulation), and the kernel turns codes into that operand on
// the way into shared memory: the codes are what crosses HBM and L2.
//
// One persistent CTA pair per two SMs (cta_group::2), a work list of (tile of G, range
// of tokens) over all layers of the call.  Tiles are 512 x 256 where they fill the
// device, else 256 x 256 (plan_batch): in the larger, two MMAs of 256 rows share a
// converted operand, which halves the conversions and their shared-memory traffic per
// flop, but their accumulators fill tensor memory, so an epilogue is not overlapped with
// the next tile's sum.
//   warp 0       TMA producer: this CTA's 128 columns of dY of each MMA, 128-byte-swizzled
//                boxes of 64 x 64 tokens (no multicast);
//   warp 1       allocates tensor memory; one lane of the leader CTA issues the MMAs;
//   warps 2-9    epilogue: tcgen05.ld, gain, shift, beta, store (or the fp32 part of a
//                range of tokens);
//   warps 10-17  converters: two groups that take k-blocks of 64 tokens in turn, codes and
//                exponent bytes from the ring of raw stages to the swizzled operand;
//   warps 18-19  fill the raw ring: codes by TMA (128 columns x 64 tokens), exponent
//                bytes (any alignment) as the aligned words that hold them by cp.async.
// Commits per k-block, to both CTAs, free dY's stage and the operand's.  The converters
// touch no global memory: the fence that shows their stores to the tensor cores waits for
// every access of the thread, and with the codes loaded by the converters themselves it
// waited for the loads of later k-blocks too (2.44 ms for 14336 x 4096 over 8192 tokens).
//
// The MMAs read the operands and write the accumulators of both CTAs, so the leader has to
// observe, at cluster scope, that the other CTA's converters have stored their half and that its
// epilogue has read the accumulator.  A release at cluster scope by the converters holds each
// up for about 1700 cycles (14336 x 4096 over 8192 tokens 828 us), by a warp that relays
// their arrivals 670 to 790 us.  So converters and epilogue arrive on barriers of their own CTA (CTA
// scope), and the other CTA's warp 1, which has no MMAs to issue, follows each completed phase with a copy of 16
// bytes into the leader's shared memory.  The copy is ordered behind what the relay has acquired, and its
// completion, counted on the leader's barrier, is a release at cluster scope, which nobody has to wait for:
// 629 us (626 with arrivals on the leader's barrier at CTA scope, which the leader need not observe).
//
// Bound by the tensor cores where there are thousands of tokens: 14336 x 4096 over 8192
// 629 us in short runs at 1965 MHz (1530 TFLOP/s; a k-block 0.80 us, of which its MMAs are 0.55), 719 us in a run of
// seconds, where the power cap holds the clock at 1395 MHz; 4096 x 4096 over 8192 190 us, over 2048 62 us (128 tiles
// for 74 pairs: a second round of parts).  fp32 dY has three bfloat16 parts to multiply: 598 us
// for 4096 x 4096 over 8192.
//
// Layers with few tiles split the tokens (plan_batch): the ranges write fp32
// parts to the workspace and a second kernel adds them in order.  768 x 768 over 16,384
// tokens: 36 us, of which the join 7; 16 layers of 2048 x 768 over 333 tokens in fp16 34 us.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <type_traits>

#include "act8.cuh"
#include "gemm.h"

namespace muon {
namespace {

constexpr int kItems = 48;              // layers per launch
constexpr int kBM = 128, kBN = 256;     // rows of one MMA in a CTA, columns of a pair's tile
constexpr int kBK = 64;                 // tokens per stage
constexpr int kBBytes = kBN / 2 * kBK * 2, kRawBytes = kBN / 2 * kBK, kExpBytes = 8 * kBK;
constexpr int kEpiWarps = 8, kConvWarps = 8, kRawWarps = 2;
constexpr int kGroupWarps = 4, kConvGroups = kConvWarps / kGroupWarps;     // converters of one k-block; k-blocks at once
constexpr int kTokens = 8 / kGroupWarps;                                   // 32-code blocks of a thread
constexpr int kThreads = 32 * (2 + kEpiWarps + kConvWarps + kRawWarps);
constexpr int kEditBytes = 2 * 4 * kBN / 2;     // fp32 gain and shift of the half of a tile's columns an epilogue warp has
constexpr int kGroup = 8;               // tile rows walked together

// MH MMAs of 256 rows share a converted operand: tiles of 256 MH x 256.
template <int MH>
struct Cfg {
    static constexpr int kABytes = MH * kBM * kBK * 2;
    static constexpr int kAStages = MH == 2 ? 3 : 6;        // dY
    static constexpr int kBStages = 4;                      // converted X^: two for the relay's way (with two 643 us)
    static constexpr int kRaw = 6;                          // codes
    static constexpr int kBufs = 2 / MH;                    // accumulators in the 512 columns
    static constexpr int kBOffset = kAStages * kABytes, kRawOffset = kBOffset + kBStages * kBBytes;
    static constexpr int kExpOffset = kRawOffset + kRaw * kRawBytes;
    static constexpr int kEditOffset = kExpOffset + kRaw * kExpBytes + 512;     // behind the barriers
    static constexpr int kSmem = 1024 + kEditOffset + kEpiWarps * kEditBytes;
    static_assert(kEpiWarps == 8 && kSmem <= 227 * 1024 && kConvGroups < kRaw, "see the converters");
    // Each stage is filled, converted, and relayed by the same warps every time.  A stage that changed hands could be
    // reached by a warp that is a phase ahead, whose wait on a parity passes at once: it would be armed twice.
    static_assert(kRaw % kRawWarps == 0 && kRaw % kConvGroups == 0 && kBStages % kConvGroups == 0, "rings");
    static_assert(16 * (kBStages + kBufs) <= 128, "the relay");
};
// The tensor cores' accumulation truncates: every 16 tokens cost up to a unit in the last place of the running sum,
// towards zero (measured 1.7e-8 relative per step, 4e-5 over 40,000 terms).  An fp32 G is therefore summed in segments of
// kSeg k-blocks, 6e-6, that are added rounded to nearest; for a 16-bit G (half a unit 2^-9 or 2^-12) 65,536
// tokens are one segment.
constexpr int kSeg32 = 96, kSeg16 = 1024;
constexpr int kPlanSms = 148;           // work lists are planned for a whole B200, so a size query needs no device

struct GradItem {
    CUtensorMap map;                    // dY: boxes of 64 columns x 64 tokens, parts as the third dimension
    CUtensorMap codes;                  // q: boxes of 128 columns x 64 tokens
    const unsigned char* e;
    long long lde;
    int rows, cols, out;
    int nkb;                            // k-blocks of one part
    int total;                          // nkb * parts
    int whole, tail;                    // tiles summed by one work item; tiles whose tokens are split into ranges
    int splits, len;                    // ranges of a tail tile (0: no tokens), k-blocks (over all parts) of one
    int tiles_m, tiles_n;
    long long begin, tail_begin;        // first entries of the work list
    void* G;
    const void *gain, *shift;
    const float* dy_sum;
    float beta;
    int vec;                            // G (and gain) rows may be accessed in 16-byte pieces; 2: fp32 in 32-byte pieces
    float* part;                        // [splits][tail][256 MH][256] fp32
};

struct GradParams {
    GradItem it[kItems];
    int n, w_dt;
    int seg;                            // k-blocks summed in tensor memory before the sum goes on in fp32 (kSeg)
    long long whole_works, works;       // whole tiles of every layer, then the ranges of the tail tiles
    int* d_status;
};

struct Work {
    int item, ti, tj;
    int kb0, kb1;                       // k-blocks
    int slot;                           // -1: a whole tile; else its part's place
};

__device__ __forceinline__ Work decode_work(const GradParams& p, long long w) {
    Work k;
    k.item = 0;
    int r;
    if (w < p.whole_works) {
        while (k.item + 1 < p.n && w >= p.it[k.item + 1].begin) ++k.item;
        r = (int)(w - p.it[k.item].begin);
        k.slot = -1;
        k.kb0 = 0;
        k.kb1 = p.it[k.item].total;
    } else {
        while (k.item + 1 < p.n && w >= p.it[k.item + 1].tail_begin) ++k.item;
        const GradItem& I = p.it[k.item];
        k.slot = (int)(w - I.tail_begin);
        const int split = k.slot / I.tail;
        r = I.whole + k.slot - split * I.tail;
        k.kb0 = split * I.len;
        k.kb1 = min(I.total, k.kb0 + I.len);
    }
    const GradItem& I = p.it[k.item];
    const int g = r / (kGroup * I.tiles_n);                 // tile rows in groups: concurrent tiles form a block
    const int gm = min(kGroup, I.tiles_m - g * kGroup);
    const int in = r - g * kGroup * I.tiles_n;
    k.ti = g * kGroup + in % gm;
    k.tj = in / gm;
    return k;
}

// A block's 32 codes to 32 16-bit values in four 16-byte pieces.
//
// The bytes of a word (four columns) are taken as two pairs of halves, columns (0, 2)
// and (1, 3), without reordering them.  Piece g of the block holds pair g of each of its
// four groups of eight columns (pairs: columns (0, 2), (1, 3), (4, 6), (5, 7) of the
// group).  That order of the operand's columns costs nothing and is the one in which a
// thread of the epilogue's 16 x 256-bit reads of the accumulator gets a whole group.
//
// Per four codes, in bfloat16: a shift and four logical operations make
// 128 + (q & 127) and the 128 or 256 to subtract (a code's sign bit is the exponent's
// lowest bit there), the difference is q and its product with 2^e is exact; in fp16
// the biased code fits the significand (1152 + q).  A bad block's codes are zeros and
// its byte the exponent of infinity: 0 * inf makes the NaNs.
template <typename T>
__device__ __forceinline__ void convert32(const uint4& a, const uint4& b, int byte, uint4 (&o)[4]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t r[4][4];
    if constexpr (IsBf16<T>::value) {
        const uint32_t scale2 = (uint32_t)byte * 0x00800080u;
        const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&scale2);
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c = w[2 * i + (g >> 1)] >> (g & 1 ? 8 : 0);
                const uint32_t v = (c & 0x007F007Fu) | 0x43004300u, d = (c & 0x00800080u) | 0x43004300u;
                const __nv_bfloat162 x = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                                         *reinterpret_cast<const __nv_bfloat162*>(&d)), s2);
                r[g][i] = *reinterpret_cast<const uint32_t*>(&x);
            }
    } else if (byte >= 127 - 24 && byte < kActFp16Top) {
        // 2^e is an fp16 value and 127 2^e in fp16's range; the product is rounded once
        const uint32_t sc = byte >= 127 - 14 ? (uint32_t)(byte - 112) << 10 : 1u << (byte - 103);
        const uint32_t scale2 = sc * 0x00010001u, off2 = 0x64806480u;
        const __half2 s2 = *reinterpret_cast<const __half2*>(&scale2), o2 = *reinterpret_cast<const __half2*>(&off2);
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c = w[2 * i + (g >> 1)] >> (g & 1 ? 8 : 0);
                const uint32_t h = (c & 0x00FF00FFu) ^ 0x64806480u;
                const __half2 x = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h), o2), s2);
                r[g][i] = *reinterpret_cast<const uint32_t*>(&x);
            }
    } else {
        // below fp16's smallest step or near the end of its range: through fp32, one rounding
        const float s = act8_step(byte);
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c = w[2 * i + (g >> 1)] >> (g & 1 ? 8 : 0);
                r[g][i] = pack2<__half>(act8_fp16((float)(signed char)c * s), act8_fp16((float)(signed char)(c >> 16) * s));
            }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) o[g] = make_uint4(r[g][0], r[g][1], r[g][2], r[g][3]);
}

// gain, shift and beta (first segment; later ones add to G) on a thread's four rows (row + 8 u) of eight columns, in the
// accumulator's register order (tmem_ld_16x256b_x4_twice, convert32).  edit: the eight columns' gain and, kBN / 2 values
// on, shift in shared memory.
template <int WDT>
__device__ __forceinline__ void edit_rows(const GradItem& I, int row, int col, bool vec, int nv, bool first, float beta,
                                          const float* edit, float (&v)[32]) {
    constexpr int at[8] = {0, 4, 1, 5, 8, 12, 9, 13};
    const int out = I.out;
    if (I.gain) {
        const float4 a = *reinterpret_cast<const float4*>(edit), b = *reinterpret_cast<const float4*>(edit + 4);
        const float g[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[16 * (u >> 1) + 2 * (u & 1) + at[i]] *= g[i];
    }
    if (I.shift && first) {
        const float4 a = *reinterpret_cast<const float4*>(edit + kBN / 2);
        const float4 b = *reinterpret_cast<const float4*>(edit + kBN / 2 + 4);
        const float s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float d = row + 8 * u < out ? I.dy_sum[row + 8 * u] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float& x = v[16 * (u >> 1) + 2 * (u & 1) + at[i]];
                x = fmaf(d, s[i], x);
            }
        }
    }
    if (beta != 0.f) {
        const long long at_row = (long long)row * I.cols + col, step = 8LL * I.cols;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Raw8<WDT> raw[2];                   // two rows' loads in flight together (four would spill)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                raw[k].load(static_cast<const char*>(I.G) + (at_row + (2 * h + k) * step) * (WDT == DT_FP32 ? 4 : 2),
                            vec && row + 8 * (2 * h + k) < out);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int u = 2 * h + k;
                float g[8];
                raw[k].get(g);
                if (!vec) load8_dt(I.G, at_row + u * step, WDT, false, row + 8 * u < out ? nv : 0, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float& x = v[16 * (u >> 1) + 2 * (u & 1) + at[i]];
                    x = fmaf(beta, g[i], x);
                }
            }
        }
    }
}

// Adds four values to memory, each rounded to nearest (subnormal sums become zeros).
__device__ __forceinline__ void red_add4(float* p, float a, float b, float c, float d) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

template <typename T, int MH, int WDT>
__global__ void __launch_bounds__(kThreads, 1) act8_grad_kernel(const __grid_constant__ GradParams p) {
    using C = Cfg<MH>;
    constexpr int kABytes = C::kABytes, kAStages = C::kAStages, kBStages = C::kBStages, kRaw = C::kRaw, kBufs = C::kBufs;
    constexpr int kBOffset = C::kBOffset, kRawOffset = C::kRawOffset, kExpOffset = C::kExpOffset;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* raw = smem + kRawOffset;
    uint64_t* afull_bar = reinterpret_cast<uint64_t*>(smem + kExpOffset + kRaw * kExpBytes);
    uint64_t* adone_bar = afull_bar + kAStages;         // the MMAs that read this stage are complete
    uint64_t* bfull_bar = adone_bar + kAStages;         // this CTA's half of an operand is converted
    uint64_t* bpeer_bar = bfull_bar + kBStages;         // leader: the other CTA's half
    uint64_t* bdone_bar = bpeer_bar + kBStages;
    uint64_t* rfull_bar = bdone_bar + kBStages;
    uint64_t* rempty_bar = rfull_bar + kRaw;
    uint64_t* tfull_bar = rempty_bar + kRaw;
    uint64_t* tempty_bar = tfull_bar + 2;
    uint64_t* drain_bar = tempty_bar + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint8_t* const relayed = smem + kExpOffset + kRaw * kExpBytes + 384;    // leader: 16 bytes per relayed barrier
    // warp and rank in forms the compiler knows to be uniform: the MMA issuer's descriptors then stay in uniform
    // registers
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;      // rank in the cluster of two
    const long long unit = blockIdx.x >> 1, nunits = gridDim.x >> 1;
    int* d_status = p.d_status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kAStages; ++s) {
            mbar_init(&afull_bar[s], 1);
            mbar_init(&adone_bar[s], 1);
        }
        for (int s = 0; s < kBStages; ++s) {
            mbar_init(&bfull_bar[s], kGroupWarps);
            mbar_init(&bpeer_bar[s], 1);                    // the armed byte count
            mbar_init(&bdone_bar[s], 1);
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(&rfull_bar[s], 33);                   // the armed byte count, each lane's exponent bytes
            mbar_init(&rempty_bar[s], kGroupWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], kEpiWarps + (rank == 0 ? 1 : 0));    // leader: and the armed byte count
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (rank == 0) {
            for (int s = 0; s < kBStages; ++s) mbar_arrive_expect_tx(&bpeer_bar[s], 16);
            for (int b = 0; b < kBufs; ++b) mbar_arrive_expect_tx(&tempty_bar[b], 16);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0;
            for (long long w = unit; w < p.works && !*abort_flag; w += nunits) {
                const Work k = decode_work(p, w);
                const GradItem& I = p.it[k.item];
                const int col = k.ti * MH * 2 * kBM + (int)rank * kBM;
                for (int kb = k.kb0; kb < k.kb1; ++kb) {
                    if (!mbar_wait<true>(&adone_bar[stage], phase ^ 1, abort_flag, d_status)) break;
                    uint8_t* sa = smem + stage * kABytes;
                    if (rank == 0) mbar_arrive_expect_tx(&afull_bar[stage], 2 * kABytes);
                    const uint32_t fb = mapa_shared(smem_u32(&afull_bar[stage]), 0);
                    const int part = kb / I.nkb, tok = (kb - part * I.nkb) * kBK;
#pragma unroll
                    for (int h = 0; h < 2 * MH; ++h)     // halves of this CTA's 128 rows of each MMA
                        tma_load_3d_pair(&I.map, fb, sa + h * (64 * kBK * 2), col + (h >> 1) * (2 * kBM) + (h & 1) * 64, tok, part);
                    if (++stage == kAStages) { stage = 0; phase ^= 1; }
                }
            }
            if (*abort_flag) {      // give the copies in flight time to land before the CTA exits
                const unsigned long long t0 = global_ns();
                while (global_ns() - t0 < 200000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------ MMA issuer
            // The whole warp walks the loop and one lane issues, so that descriptors are uniform values: with a
            // single thread in the loop each MMA took about 90 cycles to issue and a k-block about 900 of the 512
            // that its MMAs run.
            constexpr uint32_t idesc = make_idesc_f16(IsBf16<T>::value ? 1 : 0, 1, 2 * kBM, kBN) | 1u << 15;
            // start addresses stay below the descriptor's 14-bit address field, so stages are plain additions
            const uint64_t desc_a = smem_desc_sw128(smem_u32(smem), 64 * kBK * 2, 1024);
            const uint64_t desc_b = smem_desc_sw128(smem_u32(smem + kBOffset), 64 * kBK * 2, 1024);
            int as = 0, bs = 0, it = 0;
            uint32_t aphase = 0, bphase = 0;
            bool ok = true;
            for (long long w = unit; ok && w < p.works; w += nunits) {
              const Work k = decode_work(p, w);
              for (int s0 = k.kb0; ok && s0 < k.kb1; s0 += p.seg, ++it) {
                const int s1 = min(k.kb1, s0 + p.seg), buf = it % kBufs;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait<true>(&tempty_bar[buf], ((it / kBufs) & 1) ^ 1, abort_flag, d_status));
                if (!ok) break;
                if (it >= kBufs && lane == 0) mbar_arrive_expect_tx(&tempty_bar[buf], 16);     // the next reads of this accumulator
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(buf * kBN);
                for (int kb = s0; kb < s1; ++kb) {
                    bool ready = mbar_try_wait<true>(&afull_bar[as], aphase) && mbar_try_wait(&bfull_bar[bs], bphase) &&
                                 mbar_try_wait<true>(&bpeer_bar[bs], bphase);
                    if (!__all_sync(0xFFFFFFFFu, ready)) {
                        ready = mbar_wait<true>(&afull_bar[as], aphase, abort_flag, d_status) &&
                                mbar_wait(&bfull_bar[bs], bphase, abort_flag, d_status) &&
                                mbar_wait<true>(&bpeer_bar[bs], bphase, abort_flag, d_status);
                        if (!__all_sync(0xFFFFFFFFu, ready)) { ok = false; break; }
                    }
                    tc_fence_after();
                    if (lane == 0) mbar_arrive_expect_tx(&bpeer_bar[bs], 16);      // the stage's next k-block
                    // 16 tokens of an MMA: 16 rows of 128 bytes in each 64-wide box
                    const uint64_t da = desc_a + (uint64_t)(as * (kABytes >> 4)), db = desc_b + (uint64_t)(bs * (kBBytes >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < kBK / 16; ++s)
#pragma unroll
                            for (int h = 0; h < MH; ++h)
                                tc_mma_f16_pair(d_tmem + h * kBN, da + (h * kBM * kBK * 2 >> 4) + s * (2048 >> 4),
                                                db + s * (2048 >> 4), idesc, kb > s0 || s > 0 ? 1u : 0u);
                        tc_commit_pair_multicast(smem_u32(&adone_bar[as]), 3);
                        tc_commit_pair_multicast(smem_u32(&bdone_bar[bs]), 3);
                    }
                    __syncwarp();
                    if (++as == kAStages) { as = 0; aphase ^= 1; }
                    if (++bs == kBStages) { bs = 0; bphase ^= 1; }
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair_multicast(smem_u32(&tfull_bar[buf]), 3);
                __syncwarp();
              }
            }
            // no MMA may still be writing tensor memory when it is freed
            if (elect_one()) tc_commit_pair(smem_u32(drain_bar));
            __syncwarp();
            const unsigned long long t0 = global_ns();
            while (!mbar_try_wait(drain_bar, 0) && global_ns() - t0 < kWaitLimitNs) {
            }
        } else {
            // ------------------------------------------------ relay
            // Lane s < kBStages: operand stage s; the next kBufs lanes: accumulators.  Each passes the phases of a barrier of this
            // CTA on to the leader's in order, as many as there are in this CTA's work list, but for the last reads of each
            // accumulator, which nothing waits for.
            const bool op = lane < kBStages, mine = lane < kBStages + kBufs;
            const int s = op ? lane : mine ? lane - kBStages : 0;
            uint64_t* const from = op ? &bfull_bar[s] : &tempty_bar[s];
            const uint32_t to = mapa_shared(smem_u32(op ? &bpeer_bar[s] : &tempty_bar[s]), 0);
            const uint32_t slot = mapa_shared(smem_u32(relayed + 16 * (mine ? lane : 0)), 0);
            const uint8_t* const src = op ? smem + kBOffset + s * kBBytes : relayed;    // the operand's own first bytes; unused ones
            uint32_t j = s, parity = 0, blocks = 0, segs = 0, idle = 0;
            long long w = unit;
            unsigned long long t0 = 0;
            for (;;) {
                // the work list as far as the lane that is furthest along needs it
                while (w < p.works && __any_sync(0xFFFFFFFFu, mine && (op ? j >= blocks : j + kBufs >= segs))) {
                    const Work k = decode_work(p, w);
                    blocks += (uint32_t)(k.kb1 - k.kb0);
                    segs += (uint32_t)((k.kb1 - k.kb0 + p.seg - 1) / p.seg);
                    w += nunits;
                }
                const bool left = mine && (op ? j < blocks : j + kBufs < segs);
                if (!__any_sync(0xFFFFFFFFu, left)) break;
                const bool ready = left && mbar_test_wait(from, parity);
                if (ready) {
                    bulk_copy16_cluster(slot, src, to);
                    j += op ? kBStages : kBufs;
                    parity ^= 1;
                }
                if (__any_sync(0xFFFFFFFFu, ready)) {
                    idle = 0;
                } else if ((++idle & 255u) == 0) {
                    if (idle == 256u) t0 = global_ns();
                    const bool late = global_ns() - t0 > kWaitLimitNs;
                    if (late) {
                        *abort_flag = 1;
                        if (d_status && lane == 0) atomicOr(d_status, MUON_FLAG_TIMEOUT);
                    }
                    if (__any_sync(0xFFFFFFFFu, late || *abort_flag)) break;
                }
            }
            if (*abort_flag && lane == 0) {     // the copies in flight
                const unsigned long long t1 = global_ns();
                while (global_ns() - t1 < 200000ull) {
                }
            }
        }
    } else if (warp < 2 + kEpiWarps) {
        // ---------------------------------------------------- epilogue
        const int quad = warp & 3, part = (warp - 2) >> 2;
        float* const mine = reinterpret_cast<float*>(smem + C::kEditOffset + (warp - 2) * kEditBytes);
        int it = 0;
        bool ok = true;
        for (long long w = unit; ok && w < p.works; w += nunits) {
          const Work k = decode_work(p, w);
          const GradItem& I = p.it[k.item];
          // The warp's columns of gain and shift, read while the tile is summed (4096 x 4096 over 2048 tokens, bf16:
          // 62 us without them, 69 us with both, 9 us more where every 32 columns of the epilogue read theirs).
          if (k.slot < 0 && (I.gain || I.shift)) {
              __syncwarp();
#pragma unroll
              for (int i = 0; i < kBN / 64; ++i) {
                  const int col = k.tj * kBN + (2 * i + part) * 32 + lane;
                  if (I.gain) mine[i * 32 + lane] = col < I.cols ? ld_elem(I.gain, col, WDT) : 0.f;
                  if (I.shift) mine[kBN / 2 + i * 32 + lane] = col < I.cols ? ld_elem(I.shift, col, WDT) : 0.f;
              }
              __syncwarp();
          }
          for (int s0 = k.kb0; s0 < k.kb1; s0 += p.seg, ++it) {
            const int buf = it % kBufs;
            if (!mbar_wait<true>(&tfull_bar[buf], (it / kBufs) & 1, abort_flag, d_status)) { ok = false; break; }
            tc_fence_after();
            const bool first = s0 == k.kb0;         // later segments are added to G
            // the layer's fields in registers: the loop's fences would have them read again for every row
            const int out = I.out, cols = I.cols;
            const bool whole = k.slot < 0;
            const float beta = first ? I.beta : 1.f;
            const bool wide = !whole || I.vec;
            // An fp32 G that is added to as it is: by reductions in L2, which the epilogue need not wait for.  Each element
            // has one thread, whose segments' reductions keep their order.  14336 x 4096 over 8192 tokens (two segments)
            // with beta = 1 948 us with loads, 774 us so.
            const bool add_tile = WDT == DT_FP32 && whole && wide && beta == 1.f;
            const bool full = !whole || I.vec == 2;             // fp32 rows in 32-byte pieces
            const bool edit = whole && (I.gain || I.shift || beta != 0.f);
            // G, or the part's own 256 MH x 256 tile
            const int width = whole ? cols : kBN, esz = whole ? (WDT == DT_FP32 ? 4 : 2) : 4;
            const int row_at = whole ? k.ti * MH * 2 * kBM : 0, col_at = whole ? k.tj * kBN : 0;
            char* const base = whole ? static_cast<char*>(I.G)
                                     : reinterpret_cast<char*>(I.part + (long long)k.slot * (MH * 2 * kBM * kBN));
            const long long step = 8LL * width * esz;
            // A 16-bit G that is added to: the next 32 columns' values are requested before these are stored, in a loop of
            // its own for its registers (14336 x 4096 over 8192 tokens with beta 628 us, 734 us with each load waited for).
            const bool ahead = WDT != DT_FP32 && whole && I.vec && beta != 0.f;
            Raw8<DT_BF16> g[4];
            auto fetch = [&](int c) {
                const int h = c / (kBN / 32), col = k.tj * kBN + c % (kBN / 32) * 32 + (lane & 3) * 8;
                const int row = k.ti * MH * 2 * kBM + h * 2 * kBM + (int)rank * kBM + quad * 32 + (lane >> 2);
                const char* at = static_cast<const char*>(I.G) + ((long long)row * cols + col) * 2;
#pragma unroll
                for (int u = 0; u < 4; ++u, at += 16LL * cols)
                    g[u].load(at, c < MH * (kBN / 32) && col + 8 <= cols && row + 8 * u < out);
            };
            auto finish = [&](auto kind) {
            constexpr bool AHEAD = decltype(kind)::value;
            if constexpr (AHEAD) { fetch(part); }
#pragma unroll 1
            for (int c = part; c < MH * (kBN / 32); c += kEpiWarps / 4) {
                // 32 rows and 32 columns; a thread has four rows (row0 + lane / 4 + 8 u) of one group of eight columns
                // (convert32), four lanes 64 bytes or more of a row
                const int h = c / (kBN / 32), lc = c % (kBN / 32) * 32, c0 = k.tj * kBN + lc;
                const int lr = h * 2 * kBM + (int)rank * kBM + quad * 32, row0 = k.ti * MH * 2 * kBM + lr;
                if (c0 >= cols || row0 >= out) {                     // uniform over the warp
                    if constexpr (AHEAD) { fetch(c + kEpiWarps / 4); }
                    continue;
                }
                const int rows = out - row0 - (lane >> 2), nv = whole ? max(0, min(8, cols - c0 - (lane & 3) * 8)) : 8;
                const bool vec = wide && nv == 8;
                char* dst = base + ((long long)(row_at + lr + (lane >> 2)) * width + col_at + lc + (lane & 3) * 8) * esz;
                const bool add = add_tile && __all_sync(0xFFFFFFFFu, nv == 8);
                float v[32];
                tmem_ld_16x256b_x4_twice(tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)((buf + h) * kBN + lc), v);
                if (edit)
                    edit_rows<WDT>(I, row0 + (lane >> 2), c0 + (lane & 3) * 8, vec, nv, first, AHEAD || add ? 0.f : beta,
                                   mine + (lc >> 6) * 32 + (lane & 3) * 8, v);
                if constexpr (AHEAD) {                               // eight columns or none
                    constexpr int at[8] = {0, 4, 1, 5, 8, 12, 9, 13};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t w[4] = {g[u].w[0].x, g[u].w[0].y, g[u].w[0].z, g[u].w[0].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float& x0 = v[16 * (u >> 1) + 2 * (u & 1) + at[2 * i]];
                            float& x1 = v[16 * (u >> 1) + 2 * (u & 1) + at[2 * i + 1]];
                            if constexpr (WDT == DT_FP16) {
                                x0 = fmaf(beta, unpack_lo<__half>(w[i]), x0);
                                x1 = fmaf(beta, unpack_hi<__half>(w[i]), x1);
                            } else {
                                x0 = fmaf(beta, __uint_as_float(w[i] << 16), x0);
                                x1 = fmaf(beta, __uint_as_float(w[i] & 0xFFFF0000u), x1);
                            }
                        }
                    }
                    fetch(c + kEpiWarps / 4);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u, dst += step) {
                    const int z = 16 * (u >> 1) + 2 * (u & 1);
                    const float x[8] = {v[z], v[z + 4], v[z + 1], v[z + 5], v[z + 8], v[z + 12], v[z + 9], v[z + 13]};
                    if (WDT == DT_FP32 && add) {
                        // lanes exchange halves with their neighbours: each reduction covers whole sectors
                        const bool odd = lane & 1;
                        float y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = __shfl_xor_sync(0xFFFFFFFFu, odd ? x[i] : x[4 + i], 1);
                        float* at = reinterpret_cast<float*>(dst) - (odd ? 4 : 0);
                        if (8 * u < rows) {
                            red_add4(at, odd ? y[0] : x[0], odd ? y[1] : x[1], odd ? y[2] : x[2], odd ? y[3] : x[3]);
                            red_add4(at + 8, odd ? x[4] : y[0], odd ? x[5] : y[1], odd ? x[6] : y[2], odd ? x[7] : y[3]);
                        }
                        continue;
                    }
                    if (8 * u >= rows) continue;
                    // (14336 x 4096 over 8192 tokens 855 us with 16-byte stores, 747 us so)
                    if (WDT == DT_FP32 ? full && nv == 8 : !whole) {
                        Raw8<DT_FP32> o;
                        o.set(x);
                        o.store(dst, true, true);
                    } else {
                        store8_dt(dst, 0, WDT, vec, nv, x);
                    }
                }
            }
            };
            if constexpr (WDT != DT_FP32) {
                if (ahead) finish(std::true_type{});
                else finish(std::false_type{});
            } else {
                finish(std::false_type{});
            }
            tc_fence_before();
            __syncwarp();
            // only this warp's accumulator reads have to be over, not its stores
            if (lane == 0) mbar_arrive(&tempty_bar[buf]);
          }
        }
    } else if (warp < 2 + kEpiWarps + kConvWarps) {
        // ---------------------------------------------------- converters
        // Groups of kGroupWarps warps take k-blocks in turn.  A k-block is converted in registers before its stage is
        // waited for: the stage is only held for the stores, the relay and the MMAs.
        const int cw = warp - 2 - kEpiWarps, group = cw / kGroupWarps, sub = cw % kGroupWarps;
        constexpr int kTokStep = 64 / kTokens;
        // a warp: two blocks (one 64-column box of the operand), tokens tok0 + kTokStep i
        // Lanes 8 i .. 8 i + 7 hold both blocks of tokens 0, 1, 6, 7 (or 2, 3, 4, 5) of eight: their 16-byte loads of codes
        // (row = token, pieces XORed with the token's low bits: pieces {0, 2} ^ token) and their 16-byte stores
        // (pieces {0, 4} ^ token) each cover the eight bank groups.
        const int box = sub & 1, blk = lane & 1, tl = (lane >> 1) & 3;
        const int tok0 = (sub >> 1) * 16 + (lane >> 4) * 8 + ((tl < 2 ? tl : tl + 4) ^ ((lane >> 2) & 2)), x = tok0 & 7;
        const int at = kBOffset + box * (64 * kBK * 2) + tok0 * 128;
        const int codes_at = tok0 * 128, codes0 = ((box * 4 + blk * 2) ^ x) << 4, codes1 = ((box * 4 + blk * 2 + 1) ^ x) << 4;
        uint32_t rs = group, rphase = 0;                    // raw stage of the group's next k-block
        uint32_t bs = group, bphase = 1;                    // operand stage of the group's next k-block
        uint32_t n = 0, j = group;                          // k-blocks of this CTA before this work item; the group's next
        bool ok = true;
        for (long long w = unit; ok && w < p.works; w += nunits) {
            const Work k = decode_work(p, w);
            const GradItem& I = p.it[k.item];
            n += (uint32_t)(k.kb1 - k.kb0);
            // byte offset of the tokens' first exponent in its aligned word: kTokStep and kBK are multiples of 4
            const uint32_t off = ((uint32_t)reinterpret_cast<uintptr_t>(I.e) + (uint32_t)(k.tj * (kBN / kActBlock)) +
                                  rank * (kBN / 2 / kActBlock) + tok0 * (uint32_t)I.lde) & 3u;
            const int exp_at = tok0 * 8 + (int)off + box * 2 + blk;
            for (; j < n; j += kConvGroups) {
                if (!mbar_wait(&rfull_bar[rs], rphase, abort_flag, d_status)) { ok = false; break; }
                const uint8_t *r = raw + rs * kRawBytes, *e = smem + kExpOffset + rs * kExpBytes;
                uint4 o[kTokens][4];
#pragma unroll
                for (int i = 0; i < kTokens; ++i) {
                    const uint8_t* q = r + codes_at + i * (kTokStep * 128);
                    convert32<T>(*reinterpret_cast<const uint4*>(q + codes0), *reinterpret_cast<const uint4*>(q + codes1),
                                 e[exp_at + i * (kTokStep * 8)], o[i]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&rempty_bar[rs]);
                if ((rs += kConvGroups) >= kRaw) { rs -= kRaw; rphase ^= 1; }
                // the MMAs that read this operand stage last (none before its first k-block)
                if (!mbar_wait<true>(&bdone_bar[bs], bphase, abort_flag, d_status)) { ok = false; break; }
                uint8_t* const b = smem + at + bs * kBBytes;
#pragma unroll
                for (int i = 0; i < kTokens; ++i)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<uint4*>(b + i * (kTokStep * 128) + (((blk * 4 + g) ^ x) << 4)) = o[i][g];
                fence_proxy_async_smem();                   // the tensor cores read what was stored here
                __syncwarp();
                if (lane == 0) mbar_arrive(&bfull_bar[bs]);
                if ((bs += kConvGroups) >= kBStages) { bs -= kBStages; bphase ^= 1; }
            }
        }
    } else {
        // ---------------------------------------------------- raw producers
        // kRawWarps warps take k-blocks in turn: the 64 rows' exponent bytes are scattered words, whose requests
        // take one warp about as long as a k-block's MMAs.
        const uint32_t mine = warp - 2 - kEpiWarps - kConvWarps;
        uint32_t n = 0;
        bool ok = true;
        for (long long w = unit; ok && w < p.works; w += nunits) {
            const Work k = decode_work(p, w);
            const GradItem& I = p.it[k.item];
            const int col = k.tj * kBN + (int)rank * (kBN / 2), b0 = col / kActBlock;
            const int nb = min(4, act8_blocks(I.cols) - b0);            // exponent bytes of a token, if any
            const int kb0 = k.kb0;
            const uint32_t len = (uint32_t)(k.kb1 - kb0);
            uint32_t j = n + (mine + kRawWarps - n % kRawWarps) % kRawWarps;
            int tok = ((kb0 + (int)(j - n)) % I.nkb) * kBK;
            const unsigned char* src = I.e + (long long)(tok + lane) * I.lde + b0;
            const long long half = 32 * I.lde, wrap = (long long)I.nkb * kBK * I.lde;
            for (; j < n + len; j += kRawWarps) {
                const uint32_t rs = j % kRaw;
                if (!mbar_wait(&rempty_bar[rs], ((j / kRaw) & 1) ^ 1, abort_flag, d_status)) ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                uint8_t* r = raw + rs * kRawBytes;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&rfull_bar[rs], kRawBytes);
                    tma_load_3d(&I.codes, &rfull_bar[rs], r, col, tok, 0);
                }
                // The aligned words that hold a token's bytes (the second only where they cross into it);
                // tokens and columns past the end get zeros, which stand for finite values times zero codes.
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = tok + lane + 32 * h < I.rows && nb > 0;
                    const uintptr_t at = reinterpret_cast<uintptr_t>(src + h * half);
                    const int off = (int)(at & 3);
                    const char* word = reinterpret_cast<const char*>(in ? at - off : reinterpret_cast<uintptr_t>(I.e) & ~uintptr_t(3));
                    uint8_t* dst = smem + kExpOffset + rs * kExpBytes + (lane + 32 * h) * 8;
                    cp_async4(dst, word, in ? 4u : 0u);
                    if (!in) cp_async4(dst + 4, word, 0u);
                    else if (off + nb > 4) cp_async4(dst + 4, word + 4, 4u);
                }
                cp_async_mbar_arrive(&rfull_bar[rs]);
                tok += kRawWarps * kBK;
                src += kRawWarps * 2 * half;
                while (tok >= I.nkb * kBK) {                            // the next part of an fp32 dY
                    tok -= I.nkb * kBK;
                    src -= wrap;
                }
            }
            n += len;
        }
        cp_async_commit();
        cp_async_wait<0>();
        if (*abort_flag && lane == 0) {
            const unsigned long long t0 = global_ns();
            while (global_ns() - t0 < 200000ull) {
            }
        }
    }

    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// Copies of dY the tensor maps can read: rows that are not 16-byte aligned, and
// fp32 rows as three bfloat16 parts lo + mid + hi (8 significant bits each, so the
// three hold all 24; bits below 2^-133, bfloat16's smallest step, are dropped; a non-finite
// value is kept in hi), summed in that order: the small parts meet a small running sum.
// ---------------------------------------------------------------------------
struct CopyItem {
    const void* src;
    unsigned short* dst;
    long long ld, lddst, part_stride, begin;
    int rows, out, segs;
};

struct CopyParams {
    CopyItem it[kItems];
    int n;
    long long units;
};

// What the first part takes of a value: finite ones beyond bfloat16's largest, which may round to infinity, as
// that largest.  The rest, below 2^120 and a multiple of 2^104, fits the other two parts.
__device__ __forceinline__ float bf16_finite(float a) {
    const float top = __uint_as_float(0x7F7F0000u);
    return fabsf(a) > top && fabsf(a) <= 3.402823466e38f ? copysignf(top, a) : a;
}

template <int DT>
__global__ void __launch_bounds__(256) act8_copy_kernel(const __grid_constant__ CopyParams p) {
    const int lane = threadIdx.x & 31;
    const long long nwarps = (long long)gridDim.x * 8;
    int ci = 0;
    for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < p.units; u += nwarps) {
        while (ci + 1 < p.n && u >= p.it[ci + 1].begin) ++ci;
        const CopyItem& I = p.it[ci];
        const long long local = u - I.begin, row = local / I.segs;
        const int col = (int)(local - row * I.segs) * 256 + lane * 8;
        const int nv = max(0, min(8, I.out - col));
        if (nv == 0) continue;
        unsigned short* dst = I.dst + row * I.lddst + col;
        if constexpr (DT == DT_FP32) {
            const float* src = static_cast<const float*>(I.src) + row * I.ld + col;
            uint32_t o[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a = 2 * i < nv ? src[2 * i] : 0.f, b = 2 * i + 1 < nv ? src[2 * i + 1] : 0.f;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    o[k][i] = pack2<__nv_bfloat16>(bf16_finite(a), bf16_finite(b));
                    const float ra = a - unpack_lo<__nv_bfloat16>(o[k][i]), rb = b - unpack_hi<__nv_bfloat16>(o[k][i]);
                    a = fabsf(a) <= 3.402823466e38f ? ra : 0.f;
                    b = fabsf(b) <= 3.402823466e38f ? rb : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<uint4*>(dst + (2 - k) * I.part_stride) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
        } else {
            const unsigned short* src = static_cast<const unsigned short*>(I.src) + row * I.ld + col;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = 2 * i < nv ? src[2 * i] : 0u, b = 2 * i + 1 < nv ? src[2 * i + 1] : 0u;
                o[i] = a | b << 16;
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// G of the tail tiles from the parts of their token ranges (none: no tokens), added in
// order.  A warp takes a row of a tile: eight columns per lane where G's rows allow
// 16-byte accesses, else every 32nd column, so that its accesses stay together.
__global__ void __launch_bounds__(256) act8_join_kernel(const __grid_constant__ GradParams p, int tile_rows) {
    const int lane = threadIdx.x & 31;
    const long long nwarps = (long long)gridDim.x * 8;
    for (int i = 0; i < p.n; ++i) {
        const GradItem& I = p.it[i];
        const long long tile_size = (long long)tile_rows * kBN, step = I.tail * tile_size;
        const int w_dt = p.w_dt;
        for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < (long long)I.tail * tile_rows; u += nwarps) {
            const int t = (int)(u / tile_rows), lr = (int)(u - (long long)t * tile_rows), r = I.whole + t;
            const int g = r / (kGroup * I.tiles_n), gm = min(kGroup, I.tiles_m - g * kGroup), in = r - g * kGroup * I.tiles_n;
            const int row = (g * kGroup + in % gm) * tile_rows + lr, col0 = in / gm * kBN;
            if (row >= I.out) continue;
            const float* src = I.part + t * tile_size + (long long)lr * kBN;
            const float d = I.shift ? I.dy_sum[row] : 0.f;
            const long long at = (long long)row * I.cols;
            if (I.vec) {
                const int col = col0 + lane * 8;
                if (col >= I.cols) continue;
                float s[8] = {};
#pragma unroll 4
                for (int k = 0; k < I.splits; ++k) {
                    const float4 a = *reinterpret_cast<const float4*>(src + k * step + lane * 8);
                    const float4 b = *reinterpret_cast<const float4*>(src + k * step + lane * 8 + 4);
                    s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
                    s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
                }
                // fp32 rows of 8 k + 4 columns end inside a group
                const int nv = min(8, I.cols - col);
                float g8[8];
                if (I.gain) {
                    load8_dt(I.gain, col, w_dt, nv == 8, nv, g8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] *= g8[j];
                }
                if (I.shift)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] = fmaf(d, j < nv ? ld_elem(I.shift, col + j, w_dt) : 0.f, s[j]);
                if (I.beta != 0.f) {
                    load8_dt(I.G, at + col, w_dt, nv == 8, nv, g8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] = fmaf(I.beta, g8[j], s[j]);
                }
                store8_dt(I.G, at + col, w_dt, nv == 8, nv, s);
            } else {
                float s[8] = {};
#pragma unroll 2
                for (int k = 0; k < I.splits; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] += src[k * step + j * 32 + lane];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int col = col0 + j * 32 + lane;
                    if (col >= I.cols) continue;
                    float x = s[j];
                    if (I.gain) x *= ld_elem(I.gain, col, w_dt);
                    if (I.shift) x = fmaf(d, ld_elem(I.shift, col, w_dt), x);
                    if (I.beta != 0.f) x = fmaf(I.beta, ld_elem(I.G, at + col, w_dt), x);
                    st_elem(I.G, at + col, w_dt, x);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool valid(int dt) { return dt == DT_BF16 || dt == DT_FP16 || dt == DT_FP32; }

muon_status check_items(const muon_act8_grad_item* items, int n) {
    if (!items || n < 1) return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const muon_act8_grad_item& q = items[i];
        if (!act8_valid(q.c) || q.out < 1 || q.out > kActMaxDim || q.lddy < q.out || !q.G || (q.c.rows > 0 && !q.dY) ||
            !q.shift != !q.dy_sum || !std::isfinite(q.beta))
            return MUON_ERR_INVALID_ARG;
    }
    return MUON_OK;
}

// Two G's of a call that share memory would be written, and with beta read, in no order.
muon_status check_disjoint(const muon_act8_grad_item* items, int n, int w_dt) {
    struct Range { uintptr_t begin, end; };
    constexpr int kFew = 64;
    Range few[kFew];
    Range* r = n <= kFew ? few : new (std::nothrow) Range[n];
    if (!r) return MUON_ERR_UNSUPPORTED;
    for (int i = 0; i < n; ++i) {
        r[i].begin = reinterpret_cast<uintptr_t>(items[i].G);
        r[i].end = r[i].begin + (uintptr_t)items[i].out * items[i].c.cols * dt_size(w_dt);
    }
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    bool ok = true;
    for (int i = 1; i < n; ++i) ok &= r[i].begin >= r[i - 1].end;
    if (r != few) delete[] r;
    return ok ? MUON_OK : MUON_ERR_INVALID_ARG;
}

long long align256(long long x) { return (x + 255) / 256 * 256; }

// Whether the tensor map can read dY where it is.
bool direct(const muon_act8_grad_item& q, int dt) {
    return dt != DT_FP32 && rows_aligned(q.dY, q.lddy, 2) && q.lddy < (1LL << 38);
}

// Whether G's rows (and the gain) can be accessed in 16-byte pieces.
bool aligned_G(const muon_act8_grad_item& q, int w_dt) {
    return rows_aligned(q.G, q.c.cols, dt_size(w_dt)) && (reinterpret_cast<uintptr_t>(q.gain) & 15) == 0;
}

struct Plan {
    int mh;                                       // MMAs that share a converted operand: tiles of 256 mh x 256
    int whole[kItems], tail[kItems], splits[kItems], len, seg;
    long long copy_at[kItems], part_at[kItems];   // workspace offsets (-1: none)
    long long bytes;
};

// The work list.  A pair that sums a whole tile takes nkb k-blocks; the tiles run in
// rounds of 74 pairs, and a last round that is not full (or a call with fewer tiles
// than pairs) leaves pairs idle.  The tiles of that round can be split into ranges of
// tokens, shorter and fuller rounds, for fp32 parts that are written and read
// again.  Both tile sizes and every number of ranges are compared by these
// times, measured at 4096 x 4096 over 8192 tokens and 14336 x 4096 over 2048: a k-block 0.73 us with two
// MMAs per operand, 0.48 us with one (whose operand traffic per MMA is the higher), 2 us
// and 1 us per tile around its sum, parts through L2 at 3 TB/s and 4 us for the second launch.
// G whose rows cannot be written in 16-byte pieces always goes through parts: its stores are then
// whole rows of lanes instead of single elements 16 bytes apart (1000 x 777 over 300 tokens 59 us without).
void plan_batch(const muon_act8_grad_item* items, int n, int dt, int w_dt, Plan& P) {
    const int parts = dt == DT_FP32 ? 3 : 1;
    const long long pairs = kPlanSms / 2;
    bool any_unaligned = false;
    int total[kItems], longest = 0;
    for (int i = 0; i < n; ++i) {
        total[i] = (items[i].c.rows + kBK - 1) / kBK * parts;
        longest = std::max(longest, total[i]);
        any_unaligned |= !aligned_G(items[i], w_dt);
    }
    P.seg = w_dt == DT_FP32 ? kSeg32 : kSeg16;
    if (longest > P.seg) {                          // equal segments of the longest sum
        const int n_seg = (longest + P.seg - 1) / P.seg;
        P.seg = (longest + n_seg - 1) / n_seg;
    }
    double best = -1.0;
    long long best_whole = 0;
    int best_s = 1;
    P.mh = 2;
    for (int mh = 1; mh <= 2; ++mh) {
        long long tiles = 0;
        for (int i = 0; i < n; ++i)
            tiles += (long long)((items[i].out + mh * 2 * kBM - 1) / (mh * 2 * kBM)) * ((items[i].c.cols + kBN - 1) / kBN);
        const double kb_us = mh == 2 ? 0.73 : 0.48, tile_us = mh, part_us = mh * 4.0 * 2 * kBM * kBN * 2 / 3e6;
        for (int s = 1; s <= std::max((int)pairs, (longest + P.seg - 1) / P.seg) && s <= std::max(1, longest); ++s) {
            const int len = std::max(1, (longest + s - 1) / s);
            long long whole = s == 1 ? tiles : tiles / pairs * pairs;
            if (any_unaligned || (w_dt != DT_FP32 && longest > P.seg)) whole = 0;
            const long long tail = tiles - whole;
            if (tail && len > P.seg) continue;              // a part is one segment
            const double us = std::ceil((double)whole / pairs) * (longest * kb_us + tile_us * ((longest + P.seg - 1) / P.seg)) +
                              (tail ? std::ceil((double)(tail * s) / pairs) * (len * kb_us + tile_us) + tail * s * part_us + 4.0 : 0.0);
            if (best < 0.0 || us < best) {
                best = us; best_whole = whole; best_s = s; P.mh = mh;
            }
        }
    }
    P.len = std::max(1, (longest + best_s - 1) / best_s);
    P.bytes = 0;
    for (int i = 0; i < n; ++i) {
        const long long tiles = (long long)((items[i].out + P.mh * 2 * kBM - 1) / (P.mh * 2 * kBM)) *
                                ((items[i].c.cols + kBN - 1) / kBN);
        P.whole[i] = total[i] == 0 ? 0 : (int)std::min(tiles, best_whole);
        P.tail[i] = (int)(tiles - P.whole[i]);
        best_whole -= std::min(tiles, best_whole);
        P.splits[i] = (total[i] + P.len - 1) / P.len;
        P.copy_at[i] = P.part_at[i] = -1;
        if (items[i].c.rows > 0 && !direct(items[i], dt)) {
            P.copy_at[i] = P.bytes;
            P.bytes += align256(2LL * parts * items[i].c.rows * ((items[i].out + 7) / 8 * 8));
        }
        if (P.tail[i] > 0 && P.splits[i] > 0) {
            P.part_at[i] = P.bytes;
            P.bytes += 4LL * P.splits[i] * P.tail[i] * P.mh * 2 * kBM * kBN;
        }
    }
}

template <typename T, int MH, int WDT>
cudaError_t launch_one(const GradParams& prm, cudaStream_t stream) {
    constexpr int kSmem = Cfg<MH>::kSmem;
    auto kern = act8_grad_kernel<T, MH, WDT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    int dev = 0, nsm = kPlanSms;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min<long long>(prm.works, nsm / 2)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, prm);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_grad(const GradParams& prm, int dt, int mh, cudaStream_t s) {
#define ACT8_GRAD(T, MH)                                                            \
    (prm.w_dt == DT_BF16   ? launch_one<T, MH, DT_BF16>(prm, s)                     \
     : prm.w_dt == DT_FP16 ? launch_one<T, MH, DT_FP16>(prm, s) : launch_one<T, MH, DT_FP32>(prm, s))
    if (dt == DT_FP16) return mh == 2 ? ACT8_GRAD(__half, 2) : ACT8_GRAD(__half, 1);
    return mh == 2 ? ACT8_GRAD(__nv_bfloat16, 2) : ACT8_GRAD(__nv_bfloat16, 1);
#undef ACT8_GRAD
}

muon_status run_batch(const muon_act8_grad_item* items, int n, int dt, int w_dt, uint8_t* ws, int* d_status,
                      cudaStream_t stream) {
    static GradParams prm;             // large: kept off the stack, filled and consumed per launch
    static CopyParams cp;
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    Plan P;
    plan_batch(items, n, dt, w_dt, P);
    memset(&prm, 0, sizeof(prm));
    memset(&cp, 0, sizeof(cp));
    const int parts = dt == DT_FP32 ? 3 : 1;
    double flops = 0.0, copy_bytes = 0.0, join_bytes = 0.0;
    bool join = false;
    for (int i = 0; i < n; ++i) {
        const muon_act8_grad_item& q = items[i];
        GradItem& I = prm.it[i];
        I.e = q.c.e; I.lde = q.c.lde;
        I.rows = q.c.rows; I.cols = q.c.cols; I.out = q.out;
        I.nkb = (q.c.rows + kBK - 1) / kBK;
        I.total = I.nkb * parts;
        I.whole = P.whole[i];
        I.tail = P.tail[i];
        I.splits = P.splits[i];
        I.len = P.len;
        I.tiles_m = (q.out + P.mh * 2 * kBM - 1) / (P.mh * 2 * kBM);
        I.tiles_n = (q.c.cols + kBN - 1) / kBN;
        I.begin = prm.whole_works;
        prm.whole_works += I.whole;
        I.G = q.G; I.gain = q.gain; I.shift = q.shift; I.dy_sum = q.dy_sum; I.beta = q.beta;
        I.vec = !aligned_G(q, w_dt) ? 0 : (reinterpret_cast<uintptr_t>(q.G) & 31) == 0 && q.c.cols % 8 == 0 ? 2 : 1;
        I.part = P.part_at[i] < 0 ? nullptr : reinterpret_cast<float*>(ws + P.part_at[i]);
        join |= I.tail > 0;
        join_bytes += (double)I.tail * P.mh * 2 * kBM * kBN * (4.0 * I.splits + dt_size(w_dt));
        if (q.c.rows == 0) continue;
        flops += 2.0 * q.c.rows * q.out * q.c.cols;
        const void* base = q.dY;
        long long ld = q.lddy, stride = q.lddy * q.c.rows;
        if (P.copy_at[i] >= 0) {
            base = ws + P.copy_at[i];
            ld = (q.out + 7) / 8 * 8;
            stride = ld * q.c.rows;
            CopyItem& c = cp.it[cp.n++];
            c.src = q.dY; c.dst = reinterpret_cast<unsigned short*>(ws + P.copy_at[i]);
            c.ld = q.lddy; c.lddst = ld; c.part_stride = stride; c.begin = cp.units;
            c.rows = q.c.rows; c.out = q.out; c.segs = (q.out + 255) / 256;
            cp.units += (long long)c.rows * c.segs;
            copy_bytes += (double)q.c.rows * q.out * (dt_size(dt) + 2.0 * parts);
        }
        if (!tc::encode_map(&I.map, dt == DT_FP16 ? DT_FP16 : DT_BF16, base, q.out, q.c.rows, parts, ld,
                            parts == 1 ? ld : stride, 64, kBK) ||
            !tc::encode_bytes_map(&I.codes, q.c.q, q.c.cols, q.c.rows, q.c.ldq, kBN / 2, kBK))
            return MUON_ERR_CUDA;
    }
    prm.works = prm.whole_works;
    for (int i = 0; i < n; ++i) {
        prm.it[i].tail_begin = prm.works;
        prm.works += (long long)prm.it[i].tail * prm.it[i].splits;
    }
    prm.n = n;
    prm.w_dt = w_dt;
    prm.seg = P.seg;
    prm.d_status = d_status;
    int dev = 0, nsm = kPlanSms;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (cp.n > 0) {
        const int grid = (int)std::min<long long>((cp.units + 7) / 8, (long long)nsm * 8);
        trace_begin(MUON_KERNEL_ACT8, copy_bytes, stream);
        if (dt == DT_FP32) act8_copy_kernel<DT_FP32><<<grid, 256, 0, stream>>>(cp);
        else act8_copy_kernel<DT_BF16><<<grid, 256, 0, stream>>>(cp);
        trace_end(stream);
        if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
    }
    if (prm.works > 0) {
        trace_begin(MUON_KERNEL_ACT8_GRAD, flops, stream);
        const cudaError_t e = launch_grad(prm, dt, P.mh, stream);
        trace_end(stream);
        if (e != cudaSuccess) return MUON_ERR_CUDA;
    }
    if (join) {
        trace_begin(MUON_KERNEL_ACT8, join_bytes, stream);
        act8_join_kernel<<<nsm * 4, 256, 0, stream>>>(prm, P.mh * 2 * kBM);
        trace_end(stream);
        if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
    }
    return MUON_OK;
}

size_t workspace_bytes(const muon_act8_grad_item* items, int n, int dt, int w_dt) {
    long long most = 0;
    Plan P;
    for (int b = 0; b < n; b += kItems) {
        plan_batch(items + b, std::min(kItems, n - b), dt, w_dt, P);
        most = std::max(most, P.bytes);
    }
    return (size_t)most;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status act8_grad_workspace_size(const muon_act8_grad_item* items, int n, muon_dtype dy_dtype, muon_dtype w_dtype,
                                     size_t* bytes) {
    if (!bytes || !valid(dy_dtype) || !valid(w_dtype)) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_items(items, n);
    if (st != MUON_OK) return st;
    *bytes = workspace_bytes(items, n, dy_dtype, w_dtype);
    return MUON_OK;
}

muon_status act8_grad_batched(const muon_act8_grad_item* items, int n, muon_dtype dy_dtype, muon_dtype w_dtype,
                              void* workspace, size_t ws_bytes, int* d_status, muon_stream_t stream) {
    if (!valid(dy_dtype) || !valid(w_dtype)) return MUON_ERR_INVALID_ARG;
    muon_status st = check_items(items, n);
    if (st == MUON_OK) st = check_disjoint(items, n, w_dtype);
    if (st != MUON_OK) return st;
    const size_t need = workspace_bytes(items, n, dy_dtype, w_dtype);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || ws_bytes < need))
        return MUON_ERR_WORKSPACE;
    st = check_device();
    if (st != MUON_OK) return st;
    for (int b = 0; b < n; b += kItems) {
        st = run_batch(items + b, std::min(kItems, n - b), dy_dtype, w_dtype, static_cast<uint8_t*>(workspace), d_status,
                       reinterpret_cast<cudaStream_t>(stream));
        if (st != MUON_OK) return st;
    }
    return MUON_OK;
}

}  // extern "C"
