// Gradients of the layer's data movement: combine (step 4), permutation (step 2), router (step 1).
// All three are HBM streams in gather form with fp32 sums in a fixed order: no atomics, so the
// results do not depend on the schedule.
//
//   combine:   d_o[pos(t,j)] = bf16(g[t,j] * dy[t]),  d_g[t,j] = <o[pos(t,j)], dy[t]>;  shared row: dy[t]
//   permute:   dx[t] = bf16(sum_j dxs[pos(t,j)] (+ dxs[pos_shared(t)]) (+ sum_j dl[t,j] * Wr[e(t,j)]))
//   route:     s = sum_j g_j d_g_j,  dl_j = g_j (d_g_j - s);  dWr[e] = sum over e's pairs of dl * x[t],
//              db[e] = sum of dl   (the logits that were not kept have gradient zero)
#include "decode_common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace ftmoe {

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// ------------------------------------------------------------------ combine
// WPT warps per token (8 / WPT tokens per CTA; 8: a CTA of blockDim warps per token): a lane takes 16-byte
// columns, loads dy and the k rows' vectors together, writes the k scaled vectors and keeps k partial
// dot products, which a transposing reduction (nine shuffles for eight sums) and, for WPT > 1, shared
// memory finish.  KB bounds k: slots without a row cost their instructions all the same (4096 x 768,
// k = 4: 20 us with eight slots, 11 with four; 4096 x 2048, k = 6: 45 with eight, 38 with six).
template <int WPT, int KB>
__global__ void __launch_bounds__(256) combine_backward_kernel(int T, int H, int k, int S, int R,
                                                               const uint16_t* __restrict__ dy,
                                                               const uint16_t* __restrict__ o,
                                                               const int32_t* __restrict__ inv_pos,
                                                               const float* __restrict__ gw, uint16_t* __restrict__ d_o,
                                                               float* __restrict__ d_w) {
    __shared__ float part[8][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nw = WPT == 8 ? int(blockDim.x >> 5) : WPT;
    const int w = WPT == 8 ? warp : warp % WPT, tl = WPT == 8 ? 0 : warp / WPT;
    const int64_t t = int64_t(blockIdx.x) * (8 / WPT) + tl;
    float dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = 0.f;
    if (t < T) {
        int pos[KB];
        float g[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            pos[j] = -1;
            g[j] = 0.f;
            if (j < k) {
                const int p = inv_pos[t * k + j];
                pos[j] = p >= 0 && p < R ? p : -1;
                g[j] = gw[t * k + j];
            }
        }
        int ps = -1;
        if (S && d_o) {
            const int p = inv_pos[int64_t(T) * k + t];
            ps = p >= 0 && p < R ? p : -1;
        }
        const int nv = H / 8;
        for (int c = w * 32 + lane; c < nv; c += nw * 32) {
            const uint4 du = ldg_nc_v4(dy + t * H + c * 8);
            uint4 ou[KB];
            if (d_w) {
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    ou[j] = pos[j] >= 0 ? ldg_nc_v4(o + int64_t(pos[j]) * H + c * 8) : make_uint4(0, 0, 0, 0);
            }
            float d[8];
            unpack8(du, d);
            if (d_w) {
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    float x[8];
                    unpack8(ou[j], x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = fmaf(x[i], d[i], dot[j]);
                }
            }
            if (d_o) {
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (pos[j] < 0) continue;
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = g[j] * d[i];
                    *reinterpret_cast<uint4*>(d_o + int64_t(pos[j]) * H + c * 8) = pack8(x);
                }
                if (ps >= 0) *reinterpret_cast<uint4*>(d_o + int64_t(ps) * H + c * 8) = du;
            }
        }
        // a dropped pair's product with zeros is NaN where dy is not finite
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (pos[j] < 0) dot[j] = 0.f;
    }
    if (!d_w) return;
    tr_step(dot, 8, 16, lane);
    tr_step(dot, 4, 8, lane);
    tr_step(dot, 2, 4, lane);
    dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], 2);
    dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], 1);
    const int j = lane >> 2;      // the sum this lane holds (lane bits 4, 3, 2 chose the halves)
    if (WPT == 1) {
        if (t < T && (lane & 3) == 0 && j < k) d_w[t * k + j] = dot[0];
        return;
    }
    if ((lane & 3) == 0) part[warp][j] = dot[0];
    __syncthreads();
    if (t < T && w == 0 && lane < k) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WPT; ++i)
            if (i < nw) s += part[tl * WPT + i][lane];
        d_w[t * k + lane] = s;
    }
}

template <int WPT>
static void combine_backward_go(int T, int H, int k, int S, int R, const uint16_t* dy, const uint16_t* o, const int32_t* inv_pos,
                                const float* gw, uint16_t* d_o, float* d_w, cudaStream_t st) {
    const unsigned grid = unsigned((int64_t(T) * WPT + 7) / 8);
    // a CTA per token: the fewest warps that take a row in as many steps as eight would, so that few idle
    // in the last one (4096 x 2816, k = 8: 65 us with six warps, 71 with eight)
    const int pieces = (H + 255) / 256, steps = (pieces + 7) / 8;
    const int threads = WPT == 8 ? 32 * ((pieces + steps - 1) / steps) : 256;
    if (k <= 2) combine_backward_kernel<WPT, 2><<<grid, threads, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    else if (k <= 4) combine_backward_kernel<WPT, 4><<<grid, threads, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    else if (k <= 6) combine_backward_kernel<WPT, 6><<<grid, threads, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    else combine_backward_kernel<WPT, kMaxTopK><<<grid, threads, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
}

cudaError_t launch_combine_backward(int T, int H, int k, int S, int R, const uint16_t* dy, const uint16_t* o,
                                    const int32_t* inv_pos, const float* gw, uint16_t* d_o, float* d_w, cudaStream_t st) {
    // Few tokens: a CTA each (128 x 4096, k = 8: 4.8 us, 7.6 with four warps, 25.7 with one).  Long rows
    // keep it when there are more than four of them per token (8192 x 4096, k = 8: 177 us, 195 with
    // four warps), else take four (k = 4: 109, 114 with eight, 122 with one).  Short rows: a warp per token,
    // as each has a lane reduction of its own to pay (8192 x 512, k = 8: 27 us, 49 with four, 55 with
    // eight), but four while there are not enough tokens for that (512 x 1024: 4.5, 8.1 with one).
    const int w = T <= 256 || (H > 1024 && k > 4) ? 8 : H > 1024 ? 4 : T <= 1024 && H > 256 ? 4 : 1;
    if (w == 1) combine_backward_go<1>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w, st);
    else if (w == 4) combine_backward_go<4>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w, st);
    else combine_backward_go<8>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w, st);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ permutation
// One thread per 16-byte column of a token; the router's rows (fp32, two vectors per column) are
// small enough to come from L2.  KB bounds k, as above (4096 x 4096, k = 6: 56 us with eight slots, 44 with six;
// 8192 x 4096, k = 1: 49 with four, 38 with two).  Registers are held at 40 and 64, for six and four CTAs
// an SM (without a bound 8192 x 2048, k = 2 and a shared row: 27 us, with it 21; k = 8: 58.9 and 57.6).
template <bool ROUTER, int KB>
__global__ void __launch_bounds__(256, KB <= 4 ? 6 : 4) permute_backward_kernel(int T, int nv, int k, int S, int E, int R,
                                                               const uint16_t* __restrict__ dxs,
                                                               const int32_t* __restrict__ inv_pos,
                                                               const int32_t* __restrict__ idx,
                                                               const float* __restrict__ dl,
                                                               const float* __restrict__ wr, uint16_t* __restrict__ dx) {
    const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (at >= int64_t(T) * nv) return;
    const int t = int(at <= 0xFFFFFFFFll ? int64_t(uint32_t(at) / uint32_t(nv)) : at / nv);
    const int c = int(at - int64_t(t) * nv);
    uint4 u[KB + 1];
#pragma unroll
    for (int j = 0; j < KB + 1; ++j) {
        int p = -1;
        if (j < KB) { if (j < k) p = inv_pos[int64_t(t) * k + j]; }
        else if (S) p = inv_pos[int64_t(T) * k + t];
        u[j] = p >= 0 && p < R ? ldg_nc_v4(dxs + (int64_t(p) * nv + c) * 8) : make_uint4(0, 0, 0, 0);
    }
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (ROUTER) {
        // four rows of W_r in flight (with a load, its sums, then the next: 38 us for 4096 x 2048, k = 8)
        constexpr int kN = KB == 6 ? 3 : KB < 4 ? KB : 4;
        int e[KB];
        float d[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            e[j] = j < k ? idx[int64_t(t) * k + j] : -1;
            d[j] = j < k ? dl[int64_t(t) * k + j] : 0.f;
        }
#pragma unroll
        for (int j0 = 0; j0 < KB; j0 += kN) {
            float4 w[kN][2];
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int ej = e[j0 + j];
                const float4* row = reinterpret_cast<const float4*>(wr) + (int64_t(ej) * nv + c) * 2;
                const bool ok = ej >= 0 && ej < E;
                w[j][0] = ok ? __ldg(row) : make_float4(0.f, 0.f, 0.f, 0.f);
                w[j][1] = ok ? __ldg(row + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float dj = d[j0 + j];
                const float4 a = w[j][0], b = w[j][1];
                acc[0] = fmaf(dj, a.x, acc[0]); acc[1] = fmaf(dj, a.y, acc[1]); acc[2] = fmaf(dj, a.z, acc[2]); acc[3] = fmaf(dj, a.w, acc[3]);
                acc[4] = fmaf(dj, b.x, acc[4]); acc[5] = fmaf(dj, b.y, acc[5]); acc[6] = fmaf(dj, b.z, acc[6]); acc[7] = fmaf(dj, b.w, acc[7]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KB + 1; ++j) {
        float f[8];
        unpack8(u[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    *reinterpret_cast<uint4*>(dx + at * 8) = pack8(acc);
}

// The same with the router's part for many tokens: reading k fp32 rows of W_r per token from L2 moves
// twice the bytes of dx_sorted itself, so a CTA keeps W_r's 64-column slice (E x 256 bytes) in
// shared memory and takes a run of tokens through it, eight lanes a token, eight columns a lane.  The
// next tokens' positions, experts and gradients load while the current rows are summed.  Sums in the
// order of the kernel above: the same bits.  8191 tokens x 2816, k = 8, a shared row: 84 -> 76 us (504 MB,
// 6.1 TB/s); 512 threads a CTA, one CTA an SM, had left it at 96.
constexpr int kPbThreads = 256;
constexpr int kPbTokens = kPbThreads / 8;     // tokens a pass

template <int KB>
__global__ void __launch_bounds__(kPbThreads, 3) permute_backward_slice_kernel(int T, int H, int k, int S, int E, int R,
                                                                            int run, const uint16_t* __restrict__ dxs,
                                                                            const int32_t* __restrict__ inv_pos,
                                                                            const int32_t* __restrict__ idx,
                                                                            const float* __restrict__ dl,
                                                                            const float* __restrict__ wr,
                                                                            uint16_t* __restrict__ dx) {
    extern __shared__ __align__(16) float w[];      // [E][64]
    const int tid = threadIdx.x, l8 = tid & 7, col0 = blockIdx.x * 64, col = col0 + l8 * 8;
    for (int i = tid; i < E * 16; i += kPbThreads) {
        const uint32_t dst = uint32_t(__cvta_generic_to_shared(w + i * 4));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     ::"r"(dst), "l"(wr + int64_t(i >> 4) * H + col0 + (i & 15) * 4) : "memory");
    }
    const int64_t t0 = int64_t(blockIdx.y) * run;
    const int64_t end = t0 + run < T ? t0 + run : T;
    // lane j of a token's eight holds pair j: its position, expert and gradient; ps: the shared row's position
    int pos = -1, e = -1, ps = -1;
    float d = 0.f;
    const auto fetch = [&](int64_t base) {
        const int64_t t = base + (tid >> 3);
        pos = e = ps = -1;
        d = 0.f;
        if (t < end) {
            if (l8 < k) {
                pos = inv_pos[t * k + l8];
                e = idx[t * k + l8];
                d = dl[t * k + l8];
            }
            if (S) ps = inv_pos[int64_t(T) * k + t];
        }
    };
    fetch(t0);
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const int first = tid & 24;                     // the token's first lane in the warp
    for (int64_t base = t0; base < end; base += kPbTokens) {
        const int64_t t = base + (tid >> 3);
        uint4 u[KB + 1];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int p = __shfl_sync(0xffffffffu, pos, first + j);
            u[j] = p >= 0 && p < R ? ldg_nc_v4(dxs + int64_t(p) * H + col) : make_uint4(0, 0, 0, 0);
        }
        u[KB] = ps >= 0 && ps < R ? ldg_nc_v4(dxs + int64_t(ps) * H + col) : make_uint4(0, 0, 0, 0);
        const int e_now = e;
        const float d_now = d;
        fetch(base + kPbTokens);
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int ej = __shfl_sync(0xffffffffu, e_now, first + j);
            const float dj = __shfl_sync(0xffffffffu, d_now, first + j);
            const bool ok = ej >= 0 && ej < E;
            const float4* row = reinterpret_cast<const float4*>(w + (ok ? ej : 0) * 64 + l8 * 8);
            const float4 a = row[0], b = row[1];
            if (!ok) continue;
            acc[0] = fmaf(dj, a.x, acc[0]); acc[1] = fmaf(dj, a.y, acc[1]); acc[2] = fmaf(dj, a.z, acc[2]); acc[3] = fmaf(dj, a.w, acc[3]);
            acc[4] = fmaf(dj, b.x, acc[4]); acc[5] = fmaf(dj, b.y, acc[5]); acc[6] = fmaf(dj, b.z, acc[6]); acc[7] = fmaf(dj, b.w, acc[7]);
        }
#pragma unroll
        for (int j = 0; j < KB + 1; ++j) {
            float f[8];
            unpack8(u[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
        if (t < end) *reinterpret_cast<uint4*>(dx + t * H + col) = pack8(acc);
    }
}

template <int KB>
static cudaError_t permute_backward_go(int T, int H, int k, int S, int E, int R, const uint16_t* dxs, const int32_t* inv_pos,
                                       const int32_t* idx, const float* dl, const float* wr, uint16_t* dx, cudaStream_t st) {
    const int nv = H / 8;
    // Pays once dx_sorted is far larger than L2, so that W_r's rows no longer stay there: E = 128, 4096 columns,
    // 8192 tokens: k = 5 (336 MB) 89 us without, 79 with; k = 8 (537 MB) 124 and 113; but 8192 x 2048, k = 8 and
    // a shared row (302 MB), 59.2 and 60.2, with E = 256 61 and 66.  Few rows a token: 70 and 64 (k = 4, 268 MB)
    // before the register bound above, 65 since.
    if constexpr (KB > 4) {
        if (wr && (int64_t(k) + S) * T * H * 2 >= (320ll << 20)) {
            // two waves of three CTAs an SM, not a CTA more (each reads its slice of W_r once)
            const int slices = H / 64;
            int64_t runs = 6 * num_sms() / slices > 0 ? 6 * num_sms() / slices : 1;
            int64_t run = (T + runs - 1) / runs;
            run = (run + kPbTokens - 1) / kPbTokens * kPbTokens;
            runs = (T + run - 1) / run;
            const size_t smem = size_t(E) * 256;
            static PerDeviceOnce attr;
            const cudaError_t e = attr([&] {
                return cudaFuncSetAttribute(permute_backward_slice_kernel<KB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kMaxExperts * 256);
            });
            if (e != cudaSuccess) return e;
            permute_backward_slice_kernel<KB><<<dim3(slices, unsigned(runs)), kPbThreads, smem, st>>>(
                T, H, k, S, E, R, int(run), dxs, inv_pos, idx, dl, wr, dx);
            return cudaGetLastError();
        }
    }
    const int64_t blocks = (int64_t(T) * nv + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    if (wr) permute_backward_kernel<true, KB><<<unsigned(blocks), 256, 0, st>>>(T, nv, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx);
    else permute_backward_kernel<false, KB><<<unsigned(blocks), 256, 0, st>>>(T, nv, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx);
    return cudaGetLastError();
}

cudaError_t launch_permute_backward(int T, int H, int k, int S, int E, int R, const uint16_t* dxs, const int32_t* inv_pos,
                                    const int32_t* idx, const float* dl, const float* wr, uint16_t* dx, cudaStream_t st) {
    if (k <= 2) return permute_backward_go<2>(T, H, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx, st);
    if (k <= 4) return permute_backward_go<4>(T, H, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx, st);
    if (k <= 6) return permute_backward_go<6>(T, H, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx, st);
    return permute_backward_go<kMaxTopK>(T, H, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx, st);
}

// ------------------------------------------------------------------ router
struct RouteBackward {
    int T, H, k, E, P, seg, nseg;
    const uint16_t* x;
    const int32_t* idx;
    const float* gw;
    const float* dgw;
    const int32_t* offsets;
    const int32_t* sorted_flat;
    float* dlogits;
    float* dw;       // [E, H] or NULL
    float* db;       // [E] or NULL
    uint4* meta;     // [P] sorted rows: token, dlogit, expert
    float* part;     // [2 nseg, H] partial sums of experts that cross a segment border
    float* part_b;   // [2 nseg]
};

// gradient of the kept logit of flat pair p = t k + j
__device__ __forceinline__ float dlogit_of(const RouteBackward& a, int p) {
    const int t0 = p / a.k * a.k;
    float s = 0.f;
    for (int j = 0; j < a.k; ++j) s = fmaf(a.gw[t0 + j], a.dgw[t0 + j], s);
    return a.gw[p] * (a.dgw[p] - s);
}
__device__ __forceinline__ int routed_rows(const RouteBackward& a) { return max(0, min(a.offsets[a.E], a.P)); }

// Small batches (P <= kRbSmall), one launch: CTA (expert, 256 columns), the expert's rows dealt to
// eight warps, their sums joined through shared memory in warp order.  CTA e also writes the e-th
// share of dlogits.
// One launch against three, us: 6 x 128 rows at 4096 columns, E = 256: 9.9 and 13.2; 8 x 128 at 2048: 5.9 and
// 9.8; 8 x 256: 8.5 and 10.4; 8 x 512: 14.0 and 11.9.  The bound is below the crossing, as an expert's rows are one
// CTA's work here: 1024 rows in four experts 9.9 and 8.1.
constexpr int kRbSmall = 1024;

__global__ void __launch_bounds__(256) route_backward_small_kernel(RouteBackward a) {
    __shared__ float s_dl[256];
    __shared__ int s_tok[256];
    __shared__ float s_sum[8][256];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, e = blockIdx.x;
    if (blockIdx.y == 0) {
        const int share = (a.P + a.E - 1) / a.E;
        for (int i = tid; i < share; i += 256)
            if (e * share + i < a.P) a.dlogits[e * share + i] = dlogit_of(a, e * share + i);
    }
    if (!a.dw && !a.db) return;
    const int rows = routed_rows(a);
    const int lo = max(0, min(a.offsets[e], rows)), hi = max(lo, min(a.offsets[e + 1], rows));
    const int col = blockIdx.y * 256 + lane * 8;
    const bool in = a.dw && col < a.H;
    float acc[8], accb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int base = lo; base < hi; base += 256) {
        const int n = min(256, hi - base);
        __syncthreads();
        if (tid < n) {
            const int flat = a.sorted_flat[base + tid];
            const bool ok = flat >= 0 && flat < a.P;
            s_tok[tid] = ok ? flat / a.k : 0;
            s_dl[tid] = ok ? dlogit_of(a, flat) : 0.f;
        }
        __syncthreads();
        for (int r = warp; r < n; r += 32) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = in && r + 8 * i < n ? ldg_nc_v4(a.x + int64_t(s_tok[r + 8 * i]) * a.H + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (r + 8 * i >= n) break;
                const float d = s_dl[r + 8 * i];
                float f[8];
                unpack8(u[i], f);
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] = fmaf(d, f[c], acc[c]);
                accb += d;
            }
        }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) s_sum[warp][lane * 8 + c] = acc[c];
    __syncthreads();
    if (a.dw && blockIdx.y * 256 + tid < a.H) {
        float s = s_sum[0][tid];
#pragma unroll
        for (int w = 1; w < 8; ++w) s += s_sum[w][tid];
        a.dw[int64_t(e) * a.H + blockIdx.y * 256 + tid] = s;
    }
    if (a.db && blockIdx.y == 0) {
        __syncthreads();
        if (lane == 0) s_sum[0][warp] = accb;
        __syncthreads();
        if (tid == 0) {
            float s = 0.f;
            for (int w = 0; w < 8; ++w) s += s_sum[0][w];
            a.db[e] = s;
        }
    }
}

// Larger batches: the sorted order makes dWr a segmented sum over consecutive rows.  Segments are
// fixed runs of `seg` sorted rows; a CTA sums one segment for 1024 columns, expert by expert.  An
// expert that lies inside one segment is written directly; one that crosses a border leaves a partial
// sum per segment -- slot 2s (the rows at the segment's start) or 2s + 1 (the rows at its end) -- and
// the join adds them in segment order.
// Bound by L2: each of the k rows of a token is read again (8192 x 4096, k = 6: 403 MB).  Keeping a
// chunk's 64-column slice of x in shared memory reads x once, but walks rows of 128 bytes, and was
// bound by instructions (117 us with FMAs, 119 us with mma.m16n8k16 over a three-plane split, for the
// case that takes 60 us here).
__global__ void __launch_bounds__(256) route_backward_prep_kernel(RouteBackward a) {
    pdl_trigger();         // the kernel after this one reads nothing before its wait
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.P) return;
    a.dlogits[i] = dlogit_of(a, i);
    if ((!a.dw && !a.db) || i >= routed_rows(a)) return;
    const int flat = a.sorted_flat[i];
    const bool ok = flat >= 0 && flat < a.P;
    const int e = ok ? a.idx[flat] : -1;
    a.meta[i] = make_uint4(uint32_t(ok ? flat / a.k : 0), __float_as_uint(ok ? dlogit_of(a, flat) : 0.f),
                           uint32_t(e < a.E ? e : -1), 0u);
}

constexpr int kRbThreads = 128;
constexpr int kRbCols = kRbThreads * 8;
constexpr int kRbMaxSeg = 64;

__global__ void __launch_bounds__(kRbThreads) route_backward_kernel(RouteBackward a) {
    __shared__ uint4 s_m[kRbMaxSeg + 1];
    const int tid = threadIdx.x, sg = blockIdx.x, r0 = sg * a.seg;
    pdl_wait();
    pdl_trigger();
    const int n = max(0, min(a.seg, routed_rows(a) - r0));
    if (tid < n) s_m[tid] = a.meta[r0 + tid];
    if (tid == n) s_m[tid] = make_uint4(0u, 0u, 0xFFFFFFFEu, 0u);     // no row's expert: ends the last run
    __syncthreads();
    const int col = blockIdx.y * kRbCols + tid * 8;
    const bool in = a.dw && col < a.H;
    float acc[8], accb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    int run0 = 0;
    for (int b = 0; b < n; b += 8) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i] = in && b + i < n ? ldg_nc_v4(a.x + int64_t(s_m[b + i].x) * a.H + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = b + i;
            if (r >= n) break;
            const float d = __uint_as_float(s_m[r].y);
            float f[8];
            unpack8(u[i], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] = fmaf(d, f[c], acc[c]);
            accb += d;
            const int e = int(s_m[r].z);
            if (int(s_m[r + 1].z) != e) {                  // the run of this expert's rows ends here
                if (e >= 0) {
                    const bool whole = r0 + run0 == a.offsets[e] && r0 + r + 1 == a.offsets[e + 1];
                    const int slot = 2 * sg + (run0 ? 1 : 0);
                    if (in) {
                        float4* dst = reinterpret_cast<float4*>((whole ? a.dw + int64_t(e) * a.H : a.part + int64_t(slot) * a.H) + col);
                        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    }
                    if (a.db && blockIdx.y == 0 && tid == 0) *(whole ? a.db + e : a.part_b + slot) = accb;
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] = 0.f;
                accb = 0.f;
                run0 = r + 1;
            }
        }
    }
}

// Experts without rows get zeros, experts of several segments the sum of their partial sums: CTA
// (expert, 128 columns), the slots dealt to eight warps, joined in warp order.
__global__ void __launch_bounds__(256) route_backward_join_kernel(RouteBackward a) {
    __shared__ float4 s_sum[8][32];
    __shared__ float s_b[8];
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    const bool none = hi <= lo || lo < 0 || hi > a.P;
    const int s0 = none ? 0 : lo / a.seg, s1 = none ? -1 : (hi - 1) / a.seg;
    if (!none && s0 == s1) return;
    const int col = blockIdx.y * 128 + lane * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    float sb = 0.f;
#pragma unroll 4
    for (int g = s0 + warp; g <= s1; g += 8) {
        const int slot = 2 * g + (g == s0 && lo % a.seg ? 1 : 0);
        if (a.dw) {
            const float4 v = *reinterpret_cast<const float4*>(a.part + int64_t(slot) * a.H + col);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        if (a.db) sb += a.part_b[slot];
    }
    s_sum[warp][lane] = s;
    if (lane == 0) s_b[warp] = sb;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) {
        const float4 v = s_sum[w][lane];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        sb += s_b[w];
    }
    if (a.dw) *reinterpret_cast<float4*>(a.dw + int64_t(e) * a.H + col) = s;
    if (a.db && blockIdx.y == 0 && lane == 0) a.db[e] = sb;
}

// rows per segment: short ones until they fill the SMs, then longer ones (fewer partial sums).  16 against
// 64 rows, us: 6 x 680 at 4096 columns 17.2 and 20.0; 8 x 1024 at 2048 14.6 and 16.4; 6 x 2000 at 4096 28.7
// and 25.9; 8 x 2048 at 2048 20.9 and 19.0; 6 x 5460 at 4096 55.9 and 44.9
static int route_segment(int P) { return P <= 8192 ? 16 : kRbMaxSeg; }

// scratch at `part`, as laid out below; nothing for small batches
size_t route_backward_part_bytes(int T, int H, int k) {
    const int64_t P = int64_t(T) * k;
    if (P <= kRbSmall) return 0;
    const int64_t nseg = (P + route_segment(int(P)) - 1) / route_segment(int(P));
    return size_t(P) * 16 + size_t(2) * nseg * (size_t(H) + 1) * 4;
}

cudaError_t launch_route_backward(int T, int H, int k, int E, const uint16_t* x, const int32_t* idx, const float* gw,
                                  const float* dgw, const int32_t* offsets, const int32_t* sorted_flat, float* dlogits,
                                  float* dw, float* db, void* part, cudaStream_t st) {
    RouteBackward a{};
    a.T = T; a.H = H; a.k = k; a.E = E; a.P = T * k;
    a.x = x; a.idx = idx; a.gw = gw; a.dgw = dgw;
    a.offsets = offsets; a.sorted_flat = sorted_flat;
    a.dlogits = dlogits; a.dw = dw; a.db = db;
    if (a.P <= kRbSmall) {
        route_backward_small_kernel<<<dim3(E, dw ? (H + 255) / 256 : 1), 256, 0, st>>>(a);
        return cudaGetLastError();
    }
    a.seg = route_segment(a.P);
    a.nseg = (a.P + a.seg - 1) / a.seg;
    a.meta = static_cast<uint4*>(part);
    a.part = reinterpret_cast<float*>(a.meta + a.P);
    a.part_b = a.part + int64_t(2) * a.nseg * H;
    route_backward_prep_kernel<<<(a.P + 255) / 256, 256, 0, st>>>(a);
    if (dw || db) {
        cudaLaunchConfig_t cfg{};          // both start while the kernel before them drains
        cfg.gridDim = dim3(a.nseg, dw ? (H + kRbCols - 1) / kRbCols : 1);
        cfg.blockDim = dim3(kRbThreads);
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, route_backward_kernel, a);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(E, dw ? H / 128 : 1);
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, route_backward_join_kernel, a);
    }
    return cudaGetLastError();
}

}  // namespace ftmoe
