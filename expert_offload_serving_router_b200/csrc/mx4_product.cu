// Grouped product of two MXFP4 operands on the block-scaled tensor cores.
//
//   out[r, n] = sum_k a[r, k] * w[g(r), n, k]        for the rows r of each group g
//
// with the optional SwiGLU epilogue of the experts' first projection: h = silu(gate) * up from the
// fp32 accumulators, quantised to MXFP4 in the same pass (h never exists in bf16).
//
// tcgen05.mma.kind::mxf4.block_scale takes both operands as stored -- packed E2M1 codes, one E8M0
// scale per 32 elements (scale_vec::2X) -- and accumulates in fp32: every product of two E2M1 values
// and two powers of two is exact, so the only rounding before the epilogue is the accumulation's.
//
// "Weights as A": M = 128 weight rows, N = the group's rows rounded up to 16, so a group of five
// rows costs an N = 16 MMA.  Tiles are (group, at most BN rows, 128 weight rows); a group of n rows
// is cut into ceil(n / BN) nearly equal pieces.  The tile list is built by every CTA from the group
// offsets (a block scan), so nothing but the offsets has to come from the caller.
//   BN = 32:   decode batches: 8 stages of 20 KB keep 128 KB of weights in flight per SM.  Bound by HBM
//              (256 groups, 12 rows each, 4096 x 4096: 345 us, 6.7 TB/s).
//   BN = 96:   a few dozen rows a group: 6 stages of 28 KB (256 groups, 48 rows each, 2048 x 4096: 190 us, 6.4 TB/s).
//   BN = 224:  long prompts, on CTA pairs (cta_group::2, M = 256): each CTA loads 128 weight rows and half
//              of the tile's rows of `a`, 5 stages of 30 KB; two accumulators of 224 columns and two sets
//              of scale columns fill the 512 TMEM columns.  One CTA per tile moves 40 KB per 256-deep
//              stage and SM and ran at 580-600 us where pairs took 550.  256 groups x 192 rows, 4096 x 4096
//              (2.8 GB, 1.65 PFLOP): 510 us for calls a quarter of a second apart (a single launch ran at 1.50 GHz by
//              its own cycle count), 635 us back to back, where the 1 kW power cap holds the SMs at 1.07 GHz.
//
// Roles of the persistent CTA: warp 0 TMA producer (codes of both operands, 256-deep K stages, 128-byte
// swizzle); warp 1 TMEM allocator and MMA issuer; warps 2-9 read the row-major scale bytes and lay them
// out as tcgen05.cp source atoms (32 x 16 bytes per 128 rows and 128-deep K step: byte 16 (row % 32) +
// 4 (row / 32) + j = row's scale of the step's block j); warps 10-17 epilogue, two per TMEM lane quarter.
// The MMA warp copies a stage's atoms into TMEM right before the stage's MMAs (copies and MMAs of one
// thread complete in issue order).  Alone on an SM a stage of N = 192 costs 417 clocks (the MMAs 384,
// the six copies hide behind them).  Beside the other roles the issuing lane spends 380 a stage on
// copies, MMAs and commits -- the four schedulers' other warps run other code -- and waits up to 280 for data.
// Every wait is bounded.
#include "decode_common.cuh"
#include "gemm_common.cuh"
#include "mx4.cuh"
#include "mx4_tiles.h"
#include <cmath>

namespace ftmoe {

constexpr int kPxThreads = 576;
constexpr int kPxLoaders = 8;                // scale warps: two groups of four, one per chunk buffer
constexpr int kPxEpi = 8;                    // epilogue warps
constexpr int kPxK = 256;                    // K per stage: 128 bytes of codes per row
constexpr int kPxChunk = 4;                  // stages per scale chunk: 32 scale bytes of a row
constexpr int kPxSfBufs = 4;                 // chunk buffers
constexpr int kPxABytes = 128 * 128;
constexpr int kPxGroups = kMaxExperts + 1;
constexpr int kPxTable = 256;                // tiles of a CTA (pair) worked out ahead
constexpr int kPxHRow = 36;                  // fp32 per token row of an h buffer: 32 + 4 against bank conflicts

template <int BN, bool PAIR>
struct PxCfg {
    static constexpr int kStages = BN == 32 ? 8 : BN == 96 ? 6 : 5;
    static constexpr int kHalves = BN > 128 ? 2 : 1;               // 128-row scale atoms of B per 128-deep K step
    static constexpr int kBBytes = (PAIR ? BN / 2 : BN) * 128;     // a pair's CTA loads half of the rows
    static constexpr int kBox = BN == 96 ? 32 : 16;                // rows of the smallest activation box; the others are 2x, 4x
    static constexpr int kSfA = 2 * 512;
    static constexpr int kSfBytes = kSfA + 2 * kHalves * 512;      // scale atoms of one stage
    static constexpr int kSfChunk = kPxChunk * kSfBytes;           // of one chunk
    static constexpr int kSfCols = 2 * 4 + 2 * 4 * kHalves;        // TMEM columns of one stage's scales
    static constexpr int kSfBase = 2 * BN;                         // after the two accumulators
    static constexpr int kTmemCols = BN == 32 ? 128 : BN == 96 ? 256 : 512;
    static constexpr int kEpiBytes = 4 * 32 * kPxHRow * 4;         // four h buffers; >= 8 x 2 KB transpose buffers
    static constexpr size_t smem() {
        return 1024 + size_t(kStages) * (kPxABytes + kBBytes) + kPxSfBufs * kSfChunk + kEpiBytes + (2 * kStages + 2 * kPxSfBufs + 8) * 8 +
               (2 * (kPxGroups + 1) + 32) * 4 + kPxTable * 8;
    }
    static_assert(kSfBase + 2 * kSfCols <= kTmemCols, "TMEM columns");
    static_assert(kEpiBytes >= kPxEpi * kXposeBytes, "epilogue buffers");
};

struct PxParams {
    int K, nk, m_tiles, G, E, R;
    int N;                    // bf16 output columns, or weight rows per group with SwiGLU (2F)
    int vec;                  // 16: scale rows start on 16-byte boundaries; else 2
    const int32_t* offsets;
    const uint8_t* wsc;
    const uint8_t* swsc;
    const uint8_t* asc;
    uint16_t* out;
    uint8_t* hq;
    uint8_t* hs;
    uint32_t* err;
    unsigned long long wait_ns;
    int early;                // offsets and weights may be read before the wait for the preceding kernel
};

// kind::mxf4 instruction descriptor: E2M1 x E2M1, both K-major, E8M0 scales, M = 128 (256 for a
// pair); the scale ids (0 or 2) select which two of a column word's four scale bytes the 64-deep MMA takes
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (1u << 23) | (uint32_t(M >> 4) << 24) |
           (sf_id << 29);
}
template <bool PAIR>
__device__ __forceinline__ void umma_mxf4(uint32_t dtm, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t tsfa,
                                          uint32_t tsfb, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(dtm), "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(tsfa), "r"(tsfb));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(dtm), "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(tsfa), "r"(tsfb));
}
// source descriptor of a scale atom (contiguous, no swizzle) and its copy to four TMEM columns,
// repeated in every lane quarter
__device__ __forceinline__ uint64_t px_atom_desc(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t(128 >> 4) << 16 | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
}
template <bool PAIR>     // a pair's copy runs in both CTAs, each from its own shared memory to its own TMEM
__device__ __forceinline__ void px_copy_atom(uint32_t taddr, uint64_t d) {
    if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
template <bool PAIR>     // a pair's commit arrives on the barrier of both CTAs
__device__ __forceinline__ void px_commit(uint64_t* bar) {
    if constexpr (PAIR) umma_commit_pair_both(bar);
    else umma_commit(bar);
}
// the bounded wait with polls that may sleep 20 us each (a shortened bound is polled without)
static __device__ __noinline__ bool px_wait_slow(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit) {
    if (limit < kWaitNs) return mbar_wait(b, parity, abort, limit);
    const uint64_t t0 = gtimer();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(su32(b)), "r"(parity), "r"(20000u) : "memory");
        if (ok) return true;
        if (abort && *abort) return false;
        if (gtimer() - t0 > limit) return false;
    }
}
__device__ __forceinline__ bool px_wait(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit) {
    return mbar_try(b, parity) || px_wait_slow(b, parity, abort, limit);
}
__device__ __forceinline__ bool px_warp_wait(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit) {
    int r = 0;
    if ((threadIdx.x & 31) == 0) r = px_wait(b, parity, abort, limit) ? 1 : 0;
    r = __shfl_sync(0xffffffffu, r, 0);
    __syncwarp();
    return r != 0;
}
// the whole warp waits, with one outcome
__device__ __forceinline__ bool px_wait_all(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit) {
    return __all_sync(0xffffffffu, px_wait(b, parity, abort, limit)) != 0;
}
// Signals across the pair are relaxed, and what they hand over is ordered beside them: a release at cluster
// scope waits for the epilogue's global stores (2000 to 3600 clocks each time), which nobody reads here.
//   accumulators: tensor memory alone, ordered by the tcgen05 fences before the arrival and after the wait
//   scale chunks: shared memory alone, ordered by fences restricted to it (px_release_shared / px_acquire_shared)
__device__ __forceinline__ void px_arrive_peer(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void px_release_shared() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
__device__ __forceinline__ void px_acquire_shared() {
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
__device__ __forceinline__ bool px_try_peer(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(su32(b)), "r"(parity) : "memory");
    return ok != 0;
}
static __device__ __noinline__ bool px_wait_peer_slow(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit) {
    const uint64_t t0 = gtimer();
    for (uint32_t i = 1;; ++i) {
        if (px_try_peer(b, parity)) return true;
        if ((i & 31) == 0 || limit < kWaitNs) {
            if (abort && *abort) return false;
            if (gtimer() - t0 > limit) return false;
        }
    }
}
// barriers that the pair's other CTA arrives on too
template <bool PAIR>
__device__ __forceinline__ bool px_wait_peer(uint64_t* b, uint32_t parity, volatile int* abort, unsigned long long limit) {
    if constexpr (PAIR) return px_try_peer(b, parity) || px_wait_peer_slow(b, parity, abort, limit);
    else return px_wait(b, parity, abort, limit);
}
__device__ __forceinline__ bool px_elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void px_bar(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
// 16 TMEM lanes x 32 columns as mma fragments: v[4 k + i] = lane (lane / 4 + 8 (i / 2)), column 8 k + 2 (lane % 4) + i % 2
__device__ __forceinline__ void px_ld_frag(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

// silu(x) = x / (1 + 2^(-x log2 e)) to a few fp32 roundings for |x| < kPxNear -- not the tanh approximation
// of the bf16 paths: the E2M1 rounding that follows turns an error near a rounding border into a whole step.
// The exponent is carried in two floats (its rounding alone would cost |x| 2^-24), the reciprocal takes one
// Newton step.  The power is below 2^116, so nothing overflows, and flushing subnormals changes nothing: a
// subnormal exponent or power is lost in 1 + e.  NaN stays NaN.
constexpr float kPxNear = 80.f;
__device__ __forceinline__ float px_silu(float x) {
    const float n = x * -1.44269502f;                                   // log2 e = 1.44269502 + 1.92596299e-8
    const float lo = fmaf(x, -1.44269502f, -n) - x * 1.92596299e-8f;
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(n));
    const float d = 1.f + fmaf(e, lo * 0.693147182f, e);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = fmaf(r, fmaf(-d, r, 1.f), r);
    return x * r;
}
// silu(x) * u for any x, as x u / (1 + z) for x >= 0 and x z u / (1 + z) for x < 0 with z = e^-|x| <= 1, so that
// nothing overflows.  Below -kPxNear, z is kept as 2^126 z and 2^-126 multiplies u instead: a large u still
// meets it, and what then flushes (|x| > 174) is below 2^-116 whatever u is.  |x| is bounded at 190, where z u is
// zero for any u: unbounded, the exponent and its low part would grow with |x| until they overflow.  NaN
// stays NaN, +inf is inf, -inf NaN (-inf * 0), as in the formula.
__device__ __forceinline__ float px_silu_far(float x, float u) {
    const float c = fminf(fabsf(x), 190.f);
    const bool far = x < -kPxNear;
    const float n = c * -1.44269502f;
    const float lo = fmaf(c, -1.92596299e-8f, fmaf(c, -1.44269502f, -n));
    const float w = far ? 0x1p-126f : 1.f;
    float z;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(far ? n + 126.f : n));
    z = fmaf(z, lo * 0.693147182f, z);
    const float d = fmaf(z, w, 1.f);                                    // 1 .. 2
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = fmaf(r, fmaf(-d, r, 1.f), r);
    return x * r * (x < 0.f ? z : 1.f) * (u * w);
}

// 32 scale bytes (1024 elements) of a row, from byte 32 c on.  Bytes past the row's nsc are whatever
// is there: the MMAs stop at K.  Rows that start off an 8-byte boundary (K / 32 not a multiple of 8)
// are read as the aligned 8-byte words that hold them -- a word is read only if it holds a byte of the
// row, so no read leaves the allocation -- and shifted into place when they are laid out: shifting them
// here would wait for the loads.
__device__ __forceinline__ void px_load_scales(const uint8_t* row, int c, int nsc, int vec, uint64_t (&u)[5]) {
    const int o = 32 * c, n = min(32, nsc - o);
    if (vec == 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (16 * i < n) {
                const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(row + o + 16 * i);
                u[2 * i] = w.x;
                u[2 * i + 1] = w.y;
            }
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + o);
        const uint64_t* w = reinterpret_cast<const uint64_t*>(at & ~uintptr_t(7));
        const int lead = int(at & 7);
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = 8 * i < lead + n ? w[i] : 0;
    }
}
// the eight 4-byte pieces of the row at `row`
__device__ __forceinline__ void px_scale_words(const uint8_t* row, const uint64_t (&u)[5], uint32_t (&v)[8]) {
    const int sh = 8 * int(reinterpret_cast<uintptr_t>(row) & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t x = sh ? (u[i] >> sh) | (u[i + 1] << (64 - sh)) : u[i];
        v[2 * i] = uint32_t(x);
        v[2 * i + 1] = uint32_t(x >> 32);
    }
}

template <bool SWIGLU, int BN, bool PAIR>
__global__ void __launch_bounds__(kPxThreads, 1)
mx4_product_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_sw,
                   const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                   const __grid_constant__ CUtensorMap tm_a4, PxParams p) {
    using C = PxCfg<BN, PAIR>;
    constexpr int kSt = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + kSt * kPxABytes;
    uint8_t* sSf = sB + kSt * C::kBBytes;
    uint8_t* sEpi = sSf + kPxSfBufs * C::kSfChunk;
    uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + C::kEpiBytes);
    uint64_t* empty = full + kSt;
    uint64_t* tfull = empty + kSt;
    uint64_t* tempty = tfull + 2;
    uint64_t* sfull = tempty + 2;
    uint64_t* sempty = sfull + kPxSfBufs;
    uint64_t* mma_done = sempty + kPxSfBufs;
    int* ntile = reinterpret_cast<int*>(mma_done + 1);      // [G + 1] first row tile of each group
    int* off = ntile + kPxGroups + 1;                       // [G + 1] row offsets
    int* wsum = off + kPxGroups + 1;                        // block scan, then the epilogue's wait outcomes
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(wsum + 20);   // 18 warps' sums before it
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* epi_ok = abort_flag + 1;                          // [4 pairs of warps][tile parity]
    uint2* table = reinterpret_cast<uint2*>((reinterpret_cast<uintptr_t>(wsum + 30) + 7) & ~uintptr_t(7));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G;
    // tiles go to CTAs, or to pairs: the leader (rank 0) issues for both
    const int rank = PAIR ? int(cluster_ctarank()) : 0;
    const int first = PAIR ? int(blockIdx.x) >> 1 : int(blockIdx.x), stride = PAIR ? int(gridDim.x) >> 1 : int(gridDim.x);
    if (!p.early) pdl_wait();
    // ---- tile list.  A table that is not ascending in [0, R] is reported and nothing of it followed.
    int nt = 0, bad = 0;
    if (tid < G) {
        const int lo = p.offsets[tid], hi = p.offsets[tid + 1];
        bad = lo < 0 || hi < lo || hi > p.R;
        off[tid] = lo;
        if (tid == G - 1) off[G] = hi;
        nt = px_row_tiles<BN>(hi - lo);      // a bad table's are dropped below
    }
    if (__syncthreads_or(bad)) {
        if (bad && blockIdx.x == 0) atomicExch(p.err, kDevErrOffsets);
        nt = 0;
    }
    int inc = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) wsum[warp] = inc;
    if (tid == 0) {
        for (int s = 0; s < kSt; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], PAIR ? 2 * kPxEpi : kPxEpi);      // a pair's epilogue warps all arrive at the leader
        }
        for (int b = 0; b < kPxSfBufs; ++b) {
            mbar_init(&sfull[b], PAIR ? kPxLoaders : kPxLoaders / 2);      // one group's warps, in a pair of both CTAs
            mbar_init(&sempty[b], 1);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        ntile[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                         "r"(C::kTmemCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                         "r"(C::kTmemCols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    __syncthreads();
    if (tid < G) {
        for (int w = 0; w < warp; ++w) inc += wsum[w];
        ntile[tid + 1] = inc;
    }
    __syncthreads();
    const int total = ntile[G] * p.m_tiles;
    // The first kPxTable tiles of this CTA, one thread each: decoding a tile takes a search and two
    // divisions, some 1800 clocks in each of the roles' loops.
    if (tid < kPxTable && first + tid * stride < total) {
        const PxTile tl = px_tile<BN>(first + tid * stride, ntile, off, G, p.m_tiles);
        table[tid] = make_uint2(uint32_t(tl.row0), uint32_t(tl.nvalid) | uint32_t(tl.g) << 8 | uint32_t(tl.m) << 17);
    }
    const auto tile_at = [&](int t, int index) {      // tile t, this CTA's index-th
        if (index >= kPxTable) return px_tile<BN>(t, ntile, off, G, p.m_tiles);
        const uint2 e = table[index];
        return PxTile{int(e.y >> 8 & 511u), int(e.y >> 17), int(e.x), int(e.y & 255u)};
    };
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // barriers that live in the leader
    const uint32_t full_lead = PAIR ? mapa_rank(su32(full), 0) : 0u;
    const uint32_t sfull_lead = PAIR ? mapa_rank(su32(sfull), 0) : 0u;
    const uint32_t tempty_lead = PAIR ? mapa_rank(su32(tempty), 0) : 0u;
    const int nk = p.nk;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (warp-uniform, one elected lane issues)
        const int utotal = __shfl_sync(0xffffffffu, total, 0);
        const bool leader = px_elect();
        int s = 0, step = 0, j = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < utotal && ok; t += stride, ++j) {
            const PxTile tl = tile_at(t, j);
            const int g = __shfl_sync(0xffffffffu, tl.g, 0);
            const int m = __shfl_sync(0xffffffffu, PAIR ? 2 * tl.m + rank : tl.m, 0);      // 128-row weight group
            const int rows = PAIR ? ((tl.nvalid + 15) & ~15) >> 1 : tl.nvalid;                // rows of `a` this CTA loads
            const int row0 = __shfl_sync(0xffffffffu, tl.row0 + rank * rows, 0);
            const bool shared_grp = g >= p.E;
            const CUtensorMap* mw = shared_grp ? &tm_sw : &tm_w;
            const int wg = shared_grp ? 0 : g;
            // the tile's rows in units of the smallest box, loaded as at most one box of each size
            const int units = __shfl_sync(0xffffffffu, (rows + C::kBox - 1) / C::kBox, 0);
            const uint32_t bytes = uint32_t(kPxABytes) + uint32_t(units) * (C::kBox * 128u);
            const auto load_w = [&](int kb, int s) {
                uint8_t* a = sA + s * kPxABytes;
                if constexpr (PAIR) {
                    // both CTAs' bytes count on the leader's barrier, and only the leader expects them
                    if (rank == 0) mbar_expect_tx(&full[s], 2 * bytes);
                    if (SWIGLU) tma_5d_pair(mw, full_lead + 8u * s, a, kb * 128, 0, 0, m * 4, wg);
                    else tma_3d_pair(mw, full_lead + 8u * s, a, kb * 128, m * 128, wg);
                } else {
                    mbar_expect_tx(&full[s], bytes);
                    if (SWIGLU) tma_5d(mw, &full[s], a, kb * 128, 0, 0, m * 4, wg);
                    else tma_3d(mw, &full[s], a, kb * 128, m * 128, wg);
                }
            };
            const auto load_a = [&](int kb, int s) {
                uint8_t* b = sB + s * C::kBBytes;
                int r = row0;
                const auto box = [&](const CUtensorMap* tm, int n) {
                    if constexpr (PAIR) tma_2d_pair(tm, full_lead + 8u * s, b, kb * 128, r);
                    else tma_2d(tm, &full[s], b, kb * 128, r);
                    b += n * C::kBox * 128;
                    r += n * C::kBox;
                };
                if (BN > 32 && (units & 4)) box(&tm_a4, 4);
                if (units & 2) box(&tm_a2, 2);
                if (units & 1) box(&tm_a1, 1);
            };
            int early = 0;                     // stages whose weights are already on their way
            if (step == 0) {
                // the ring's first round: weights before the wait for the kernel that writes the activations
                early = min(kSt, nk);
                if (leader) {
                    for (int kb = 0; kb < early; ++kb) load_w(kb, kb);
                    pdl_wait();
                    pdl_trigger();             // after the wait: what this kernel waited for is final for its dependent too
                }
                __syncwarp();
            }
            for (int kb = 0; kb < nk; ++kb, ++step) {
                // a stage of the first round is free, and its weights may be on their way: it is always completed
                ok = kb < early || px_wait_all(&empty[s], phase ^ 1u, abort_flag, p.wait_ns);
                if (!ok) break;
                if (leader) {
                    if (kb >= early) load_w(kb, s);
                    load_a(kb, s);
                }
                __syncwarp();
                if (++s == kSt) { s = 0; phase ^= 1u; }
            }
        }
        if (leader) {
            if (!ok) { *abort_flag = 1; atomicExch(p.err, kDevErrTimeout); }
            // own copies in flight have landed: the leader sees its full barriers complete (in a pair both CTAs'
            // bytes), the peer that the leader consumed what it copied
            // (after an abort the other CTA may never bring its part: one default bound is ample for one's own)
            for (int st = step > kSt ? step - kSt : 0; st < step; ++st)
                if (!mbar_wait(rank == 0 ? &full[st % kSt] : &empty[st % kSt], uint32_t(st / kSt) & 1u, nullptr)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ scale copies and MMAs
        // One elected lane runs a tile's K loop: under elect.sync the descriptors stay in uniform registers,
        // where the tcgen05 instructions want them.  (Under `if (lane == 0)` every operand is moved there
        // one by one: 1200 clocks a stage of N = 192 against under 800 then; the whole warp looping and the
        // elected lane issuing paid a vote and a reconvergence a stage.)  The loop is unrolled by a chunk,
        // so that scale columns and atom offsets are constants: per stage 550 clocks of issue became 370
        // (one token, 6 of 256 groups, 4096 x 4096: 18.1 -> 16.6 us).
        const int utotal = rank == 0 ? __shfl_sync(0xffffffffu, total, 0) : 0;      // the leader issues for the pair
        const bool leader = px_elect();
        const uint64_t ad0 = sdesc_sw128(su32(sA)), bd0 = sdesc_sw128(su32(sB));
        const uint64_t sf0 = px_atom_desc(su32(sSf));
        int s = 0, j = 0, ch = 0;             // stage, tile and scale chunk counters
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < utotal; t += stride, ++j) {
            const PxTile tl = tile_at(t, j);
            const int N = __shfl_sync(0xffffffffu, (tl.nvalid + 15) & ~15, 0);
            const int buf = j & 1;
            ok = __all_sync(0xffffffffu, px_wait_peer<PAIR>(&tempty[buf], (uint32_t(j >> 1) & 1u) ^ 1u, abort_flag, p.wait_ns)) != 0;
            if (!ok) break;
            tc_fence_after();
            const uint32_t dacc = tmem + uint32_t(BN * buf);
            const uint32_t id0 = idesc_mxf4(PAIR ? 256 : 128, N, 0), id2 = idesc_mxf4(PAIR ? 256 : 128, N, 2);
            const bool two = C::kHalves == 2 && N > 128;
            if (leader) {
                int st = s, c = ch;
                uint32_t ph = phase;
                const int full_k = p.K / kPxK;
#pragma unroll 4
                for (int kb = 0; kb < nk; ++kb) {
                    if ((kb & (kPxChunk - 1)) == 0) {
                        ok = px_wait_peer<PAIR>(&sfull[c % kPxSfBufs], uint32_t(c / kPxSfBufs) & 1u, abort_flag, p.wait_ns);
                        if (!ok) break;
                        if constexpr (PAIR) px_acquire_shared();
                    }
                    ok = px_wait(&full[st], ph, abort_flag, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const bool chunk_end = (kb & (kPxChunk - 1)) == kPxChunk - 1 || kb == nk - 1;
                    const uint32_t sfa = tmem + uint32_t(C::kSfBase + (kb & 1) * C::kSfCols), sfb = sfa + 8u;
                    const uint64_t sd = sf0 + uint64_t(((c % kPxSfBufs) * C::kSfChunk + (kb & (kPxChunk - 1)) * C::kSfBytes) >> 4);
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        px_copy_atom<PAIR>(sfa + 4u * a, sd + uint64_t(32 * a));
                        px_copy_atom<PAIR>(sfb + 4u * C::kHalves * a, sd + uint64_t((C::kSfA + a * C::kHalves * 512) >> 4));
                        if (two) px_copy_atom<PAIR>(sfb + 4u * C::kHalves * a + 4u, sd + uint64_t((C::kSfA + a * C::kHalves * 512 + 512) >> 4));
                    }
                    const uint64_t ad = ad0 + uint64_t((st * kPxABytes) >> 4), bd = bd0 + uint64_t((st * C::kBBytes) >> 4);
                    const auto mma = [&](int i) {            // 64 deep
                        const uint32_t hi = (i & 1) ? 2u << 30 : 0u;
                        umma_mxf4<PAIR>(dacc, ad + uint64_t(2 * i), bd + uint64_t(2 * i), (i & 1) ? id2 : id0,
                                  (sfa + 4u * (i >> 1)) | hi, (sfb + 4u * C::kHalves * (i >> 1)) | hi, (kb | i) != 0);
                    };
                    if (kb < full_k) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma(i);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < ((p.K >> 6) & 3); ++i) mma(i);
                    }
                    px_commit<PAIR>(&empty[st]);
                    if (chunk_end) { px_commit<PAIR>(&sempty[c % kPxSfBufs]); ++c; }
                    if (++st == kSt) { st = 0; ph ^= 1u; }
                }
                if (ok) px_commit<PAIR>(&tfull[buf]);
            }
            ok = __all_sync(0xffffffffu, ok) != 0;
            if (!ok) break;
            ch += (nk + kPxChunk - 1) / kPxChunk;
            phase ^= uint32_t((s + nk) / kSt) & 1u;
            s = (s + nk) % kSt;
        }
        __syncwarp();
        if (leader) {
            if (!ok) { *abort_flag = 1; atomicExch(p.err, kDevErrTimeout); }
            if (rank == 0) px_commit<PAIR>(mma_done);     // completion of every MMA and copy above, in both CTAs
            mbar_wait(mma_done, 0, nullptr);
        }
        __syncwarp();
    } else if (warp < 2 + kPxLoaders) {
        // ------------------------------------------------ scale bytes -> atoms, a chunk (four stages) at a time
        // Two groups of four warps take alternate chunks, a buffer each; thread i of a group takes A row i
        // and B rows i, i + 128, 32 bytes of each.  A chunk's loads are issued right after the group's
        // last one was laid out, so they have two chunks' MMA time to arrive.  (One group took a
        // memory latency per chunk, and deeper register queues did not help: their loads share scoreboards.
        // 129 groups of 143 rows, N 1408, K 2816: 82 -> 72 us.)
        // One proxy fence and one arrival per chunk: per stage they made this warp the slowest.
        const int grp = (warp - 2) >> 2, i = (tid - 64) & 127;
        const int nsc = p.K / 32, nch = (nk + kPxChunk - 1) / kPxChunk;
        const int at = 16 * (i & 31) + 4 * (i >> 5);
        constexpr int kRows = 1 + C::kHalves;
        uint64_t raw[kRows][5] = {};
        int lt = first, lj = 0, lc = 0, cur = -1;      // the load cursor, and the tile its row pointers are of
        const uint8_t* src[kRows] = {};
        bool take[kRows] = {};
        auto advance = [&](int n) {
            for (lc += n; lc >= nch; lc -= nch, ++lj) lt += stride;
        };
        const auto weight_row = [&](const PxTile& tl) {      // this thread's A row of a tile
            const bool shared_grp = tl.g >= p.E;
            const int mg = PAIR ? 2 * tl.m + rank : tl.m;
            int wrow;
            if (SWIGLU) {
                const int F = p.N >> 1, f = min(mg * 64 + 16 * (i >> 5) + (i & 15), F - 1);
                wrow = (i & 31) < 16 ? f : F + f;
            } else {
                wrow = min(mg * 128 + i, p.N - 1);
            }
            return (shared_grp ? p.swsc : p.wsc) + (size_t(shared_grp ? 0 : tl.g) * p.N + wrow) * nsc;
        };
        auto load = [&]() {
            if (lt >= total) return;
            if (lt != cur) {
                cur = lt;
                const PxTile tl = tile_at(lt, lj);
                src[0] = weight_row(tl);
                take[0] = true;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h) {
                    take[1 + h] = i + 128 * h < ((tl.nvalid + 15) & ~15);
                    src[1 + h] = p.asc + size_t(tl.row0 + min(i + 128 * h, tl.nvalid - 1)) * nsc;
                }
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (take[r]) px_load_scales(src[r], lc, nsc, p.vec, raw[r]);
        };
        bool ok = true;
        pdl_wait();                            // the activations' scales come from the preceding kernel
        advance(grp);
        load();
        for (int ch = grp; lt < total; ch += 2) {
            const int b = ch % kPxSfBufs;
            if (!px_warp_wait(&sempty[b], (uint32_t(ch / kPxSfBufs) & 1u) ^ 1u, abort_flag, p.wait_ns)) { ok = false; break; }
            uint8_t* d = sSf + b * C::kSfChunk + at;
            uint32_t v[kRows][8];
#pragma unroll
            for (int r = 0; r < kRows; ++r) px_scale_words(src[r], raw[r], v[r]);     // src: still this chunk's tile
#pragma unroll
            for (int sub = 0; sub < kPxChunk; ++sub)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    *reinterpret_cast<uint32_t*>(d + sub * C::kSfBytes + 512 * a) = v[0][2 * sub + a];
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        *reinterpret_cast<uint32_t*>(d + sub * C::kSfBytes + C::kSfA + (a * C::kHalves + h) * 512) = v[1 + h][2 * sub + a];
                }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                if (PAIR && rank == 1) {
                    px_release_shared();
                    px_arrive_peer(sfull_lead + 8u * b);
                } else {
                    mbar_arrive(&sfull[b]);
                }
            }
            advance(2);
            load();
        }
        if (!ok) { *abort_flag = 1; if (lane == 0) atomicExch(p.err, kDevErrTimeout); }
    } else {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;                       // TMEM lanes 32q .. 32q + 31
        const int half = (warp - 2 - kPxLoaders) >> 2;   // column chunks half, half + 2, ...
        // SwiGLU: the two warps of a lane half of the accumulator share the 32 columns of h of one MXFP4 block
        const int duo = 2 * half + (q >> 1), et = 32 * (q & 1) + lane;      // pair 0..3, thread 0..63 of it
        const auto release = [&](int buf) {
            if (lane) return;
            if constexpr (PAIR) px_arrive_peer(tempty_lead + 8u * buf);
            else mbar_arrive(&tempty[buf]);
        };
        bool ok = true;
        int j = 0;
        for (int t = first; t < total; t += stride, ++j) {
            const PxTile tl = tile_at(t, j);
            const int buf = j & 1;
            const uint32_t par = uint32_t(j >> 1) & 1u;
            if (SWIGLU) {
                // the two warps meet at barriers below, so they take one common outcome
                if (!(q & 1)) {
                    const bool r = px_warp_wait(&tfull[buf], par, abort_flag, p.wait_ns);
                    if (lane == 0) epi_ok[2 * duo + buf] = r;
                    __threadfence_block();
                }
                px_bar(1 + duo);
                ok = epi_ok[2 * duo + buf] != 0;       // overwritten two tiles on, past the next tile's barrier
            } else {
                ok = px_warp_wait(&tfull[buf], par, abort_flag, p.wait_ns);
            }
            if (!ok) break;
            tc_fence_after();
            const int mg = PAIR ? 2 * tl.m + rank : tl.m;
            // a pair tile's second weight group may lie past the last one: nothing of it is stored
            const bool store = !PAIR || mg < (SWIGLU ? p.N / 128 : (p.N + 127) / 128);
            const int nch = (tl.nvalid + 31) >> 5;
            const uint32_t tb = tmem + (uint32_t(q * 32) << 16) + uint32_t(BN * buf);
            for (int c = half; c < nch; c += 2) {
                float v0[16], v1[16];                  // the warp's first and second 16 weight rows
                px_ld_frag(tb + uint32_t(32 * c), v0);
                px_ld_frag(tb + (16u << 16) + uint32_t(32 * c), v1);
                tmem_wait_16(v0);
                tmem_fence_regs(v1);
                if (c + 2 >= nch) {                    // this warp's last read of the accumulator
                    tc_fence_before();
                    __syncwarp();
                    release(buf);
                }
                if constexpr (SWIGLU) {
                    // the first 16 rows are gate rows f, the second the up rows of the same f: both in the same
                    // place of the fragment.  h is staged as fp32 [token][32 f of the pair]
                    float* hb = reinterpret_cast<float*>(sEpi) + duo * 32 * kPxHRow;
                    float* hw = hb + (lane & 3) * 2 * kPxHRow + 16 * (q & 1) + (lane >> 2);
                    const auto put = [&](int i, float h) { hw[(8 * (i >> 2) + (i & 1)) * kPxHRow + 8 * ((i >> 1) & 1)] = h; };
                    // one look at the sixteen gates: the form for any gate everywhere costs 1 % (2049 tokens, 8 of
                    // 128 + 1, 2816 x 704: 123.3 us, 122.1 with the short form where it holds)
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(v0[i]));
                    if (__builtin_expect(top < kPxNear, 1)) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) put(i, px_silu(v0[i]) * v1[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) put(i, px_silu_far(v0[i], v1[i]));
                    }
                    px_bar(1 + duo);
                    const int tok = et >> 1, part = et & 1;   // two threads per 32-element block
                    const float4* hr = reinterpret_cast<const float4*>(hb + tok * kPxHRow + 16 * part);
                    float x[16];
                    uint32_t m = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 u = hr[i];
                        x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    float mul;
                    const uint32_t sc = mx4_scale_of(m, mul);
                    float y[8], z[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) { y[i] = x[i] * mul; z[i] = x[8 + i] * mul; }
                    uint2 cd = make_uint2(e2m1x8(y), e2m1x8(z));
                    if (sc == 255u) cd = make_uint2(0u, 0u);
                    const int n = 32 * c + tok;
                    if (store && n < tl.nvalid) {
                        const int F = p.N >> 1;
                        const size_t row = size_t(tl.row0 + n);
                        *reinterpret_cast<uint2*>(p.hq + row * (F >> 1) + mg * 32 + 16 * (q >> 1) + 8 * part) = cd;
                        if (!part) p.hs[row * (F >> 5) + mg * 2 + (q >> 1)] = uint8_t(sc);
                    }
                    px_bar(1 + duo);
                } else {
                    // bf16 pairs of two tokens per weight row, stored transposed: token rows of 64 bytes, their
                    // 16-byte pieces XORed with the token so that neither side meets on a bank
                    uint8_t* xb = sEpi + (warp - 2 - kPxLoaders) * kXposeBytes;
                    const uint32_t dst = su32(xb) + uint32_t(lane & 7) * 64u + uint32_t(((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t a0 = pack_bf16x2(v0[4 * k], v0[4 * k + 1]), a1 = pack_bf16x2(v0[4 * k + 2], v0[4 * k + 3]);
                        const uint32_t a2 = pack_bf16x2(v1[4 * k], v1[4 * k + 1]), a3 = pack_bf16x2(v1[4 * k + 2], v1[4 * k + 3]);
                        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                                     ::"r"(dst + 512u * k), "r"(a0), "r"(a1), "r"(a2), "r"(a3) : "memory");
                    }
                    __syncwarp();
                    const int col = mg * 128 + 32 * q;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int ch = lane + 32 * r, tok = ch >> 2, pp = ch & 3;
                        const int n = 32 * c + tok;
                        if (n < tl.nvalid && col + 8 * pp < p.N)
                            *reinterpret_cast<uint4*>(p.out + size_t(tl.row0 + n) * p.N + col + 8 * pp) =
                                *reinterpret_cast<const uint4*>(xb + tok * 64 + ((pp ^ ((tok >> 1) & 3)) << 4));
                    }
                    __syncwarp();
                }
            }
            if (half >= nch) {                         // no chunk of this tile is this warp's
                tc_fence_before();
                __syncwarp();
                release(buf);
            }
        }
        if (!ok) { *abort_flag = 1; if (lane == 0) atomicExch(p.err, kDevErrTimeout); }
    }
    if (warp == 0) pdl_wait();     // a CTA without tiles too: the grid's end stands for all before it
    // a pair: every MMA is complete (mma_done) and both CTAs are past their last TMEM read and remote
    // arrival before the TMEM is freed and either CTA exits
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
    }
}

template <bool SWIGLU, int BN, bool PAIR>
static int launch_variant(int64_t tiles, cudaStream_t st, const CUtensorMap& tw, const CUtensorMap& tsw,
                          const CUtensorMap (&ta)[3], const PxParams& p) {
    constexpr size_t smem = PxCfg<BN, PAIR>::smem();
    static PerDeviceOnce attr;
    if (attr([&] {
            return cudaFuncSetAttribute(mx4_product_kernel<SWIGLU, BN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        }) != cudaSuccess)
        return 2;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kPxThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    if (PAIR) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    cfg.attrs = at;
    int workers = num_sms();       // persistent CTAs, or pairs: as many as fit at once
    if (PAIR) {
        static PerDeviceCount max_clusters;
        workers = max_clusters([&] {
            cfg.gridDim = dim3(2 * (num_sms() / 2));
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, mx4_product_kernel<SWIGLU, BN, PAIR>, &cfg) != cudaSuccess || n <= 0) {
                cudaGetLastError();
                n = num_sms() / 2;
            }
            return n;
        });
    }
    if (tiles < workers) workers = int(tiles);
    cfg.gridDim = dim3(PAIR ? 2 * workers : workers);
    // Always a programmatic dependent.  Behind a kernel of unknown origin everything is read after the
    // wait; behind the token quantiser or this kernel, which start dependents only after their own
    // wait and write neither offsets nor weights, those two are final and are read before it (early).
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
    return cudaLaunchKernelEx(&cfg, mx4_product_kernel<SWIGLU, BN, PAIR>, tw, tsw, ta[0], ta[1], ta[2], p) == cudaSuccess ? 0 : 2;
}

// Which tile: the persistent workers (CTAs, or pairs) take rounds of tiles, so the estimate is rounds
// times the measured time of a round, 6.5 : 8 : 12 for the three tiles (K = 4096, one round of each:
// 8.7, 10.1 and 13.8 us).  Row tiles of a group: one while its average is well inside the tile, else as
// many as the bound allows.  Measured (us, BN = 32 / 96 / pairs; the pick is the smallest of each):
//   256 groups, 2048 x 4096: 8 rows each 177 / 179 / 189, 24 183 / 184 / 194, 32 206 / 186 / 196, 97 494 / 262 / 218;
//   128 groups, 2816 x 704: 8 rows 27.8 / 29.2 / 31.3, 32 38.7 / 30.0 / 32.6, 128 111 / 55 / 42;   one group, 4096 x 4096:
//   64 rows 8.7 / 8.9 / 10.4, 200 13.4 / 10.3 / 13.8, 400 18.6 / 15.9 / 14.0, 1600 58 / 28 / 21;   1000 rows, 512 x 4096:
//   8.7 / 10.1 / 13.8.
static int pick_tile(const Mx4Launch& L, int row_groups) {
    const double groups = L.G < L.R ? L.G : L.R, avg = L.R / groups;
    const int bn[3] = {32, 96, 224};
    const double cost[3] = {6.5, 8., 12.};
    const int sms = num_sms();
    int best = 0;
    double least = 0.;
    for (int i = 0; i < 3; ++i) {
        const double tiles = groups * (avg <= 0.8 * bn[i] ? 1. : 1. + avg / bn[i]) * (i == 2 ? (row_groups + 1) / 2 : row_groups);
        const double t = cost[i] * ceil(tiles / (i == 2 ? sms / 2 : sms));
        if (i == 0 || t < least) { best = i; least = t; }
    }
    return best;
}

int launch_mx4_product(const Mx4Launch& L, cudaStream_t st) {
    const int wrows = L.swiglu ? 2 * L.N : L.N;        // weight rows per group
    const uint64_t kb = uint64_t(L.K) / 2;             // code bytes per row
    const int row_groups = L.swiglu ? L.N / 64 : (L.N + 127) / 128;      // 128-row weight groups
    const int tile = pick_tile(L, row_groups);
    const bool small = tile == 0, mid = tile == 1;
    CUtensorMap tw{}, tsw{}, ta[3]{};
    for (int i = 0; i < 3; ++i) {
        if ((small || mid) && i == 2) { ta[2] = ta[1]; break; }     // BN = 32 and 96 have two sizes
        uint64_t dims[2] = {kb, uint64_t(L.R)};
        uint64_t str[1] = {kb};
        uint32_t box[2] = {128, (mid ? 32u : 16u) << i};
        if (!make_map(&ta[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, L.a, 2, dims, str, box)) return 1;
    }
    auto weight_map = [&](CUtensorMap* m, const uint8_t* w, int groups) {
        if (L.swiglu) {
            // [E][2][F][K/2] viewed as (K/2, 16, 2, F/16, E): a box of four blocks of 16 gate rows, each
            // followed by the 16 matching up rows
            const uint64_t F = uint64_t(L.N);
            uint64_t dims[5] = {kb, 16, 2, F / 16, uint64_t(groups)};
            uint64_t str[4] = {kb, F * kb, 16 * kb, 2 * F * kb};
            uint32_t box[5] = {128, 16, 2, 4, 1};
            return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, 5, dims, str, box);
        }
        uint64_t dims[3] = {kb, uint64_t(L.N), uint64_t(groups)};
        uint64_t str[2] = {kb, uint64_t(L.N) * kb};
        uint32_t box[3] = {128, 128, 1};
        return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, 3, dims, str, box);
    };
    if (!weight_map(&tw, L.w, L.E)) return 1;
    if (L.G > L.E) {
        if (!weight_map(&tsw, L.sw, 1)) return 1;
    } else {
        tsw = tw;
    }
    PxParams p{};
    p.K = L.K;
    p.nk = (L.K + kPxK - 1) / kPxK;
    p.m_tiles = tile == 2 ? (row_groups + 1) / 2 : row_groups;           // a pair takes two
    p.G = L.G; p.E = L.E; p.R = L.R; p.N = wrows;
    p.offsets = L.offsets;
    p.wsc = L.ws; p.swsc = L.sws; p.asc = L.as;
    p.out = L.out; p.hq = L.hq; p.hs = L.hs;
    p.err = L.err;
    p.early = L.early;
    p.wait_ns = gemm_wait_ns();
    const uintptr_t al = reinterpret_cast<uintptr_t>(L.ws) | reinterpret_cast<uintptr_t>(L.as) |
                         (L.G > L.E ? reinterpret_cast<uintptr_t>(L.sws) : 0) | uintptr_t(L.K / 32);
    p.vec = al % 16 == 0 ? 16 : 2;
    const int64_t bn = small ? 32 : mid ? 96 : 224;
    const int64_t tiles = int64_t(p.m_tiles) * (int64_t(L.G < L.R ? L.G : L.R) + L.R / bn);   // an upper bound
    if (L.swiglu)
        return small ? launch_variant<true, 32, false>(tiles, st, tw, tsw, ta, p)
               : mid ? launch_variant<true, 96, false>(tiles, st, tw, tsw, ta, p)
                     : launch_variant<true, 224, true>(tiles, st, tw, tsw, ta, p);
    return small ? launch_variant<false, 32, false>(tiles, st, tw, tsw, ta, p)
           : mid ? launch_variant<false, 96, false>(tiles, st, tw, tsw, ta, p)
                 : launch_variant<false, 224, true>(tiles, st, tw, tsw, ta, p);
}

}  // namespace ftmoe
