// Gradients of the layer's data movement: combine (step 4), permutation (step 2), router (step 1).
// All three are HBM streams in gather form with fp32 sums in a fixed order: no atomics, so the
// results do not depend on the schedule.
//
//   combine:   d_o[pos(t,j)] = bf16(g[t,j] * dy[t]),  d_g[t,j] = <o[pos(t,j)], dy[t]>;  shared row: dy[t]
//   permute:   dx[t] = bf16(sum_j dxs[pos(t,j)] (+ dxs[pos_shared(t)]) (+ sum_j dl[t,j] * Wr[e(t,j)]))
//   route:     s = sum_j g_j d_g_j,  dl_j = g_j (d_g_j - s);  dWr[e] = sum over e's pairs of dl * x[t],
//              db[e] = sum of dl   (the logits that were not kept have gradient zero)
#include "kernels.h"

namespace ftmoe {

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// ------------------------------------------------------------------ combine
// WPT warps per token (8 / WPT tokens per CTA): a lane takes 16-byte columns, loads dy and the k
// rows' vectors together, writes the k scaled vectors and keeps k partial dot products, which a
// transposing reduction (nine shuffles for eight sums) and, for WPT > 1, shared memory finish.
template <int WPT>
__global__ void __launch_bounds__(256) combine_backward_kernel(int T, int H, int k, int S, int R,
                                                               const uint16_t* __restrict__ dy,
                                                               const uint16_t* __restrict__ o,
                                                               const int32_t* __restrict__ inv_pos,
                                                               const float* __restrict__ gw, uint16_t* __restrict__ d_o,
                                                               float* __restrict__ d_w) {
    __shared__ float part[8][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int w = warp % WPT, tl = warp / WPT;
    const int64_t t = int64_t(blockIdx.x) * (8 / WPT) + tl;
    float dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = 0.f;
    if (t < T) {
        int pos[kMaxTopK];
        float g[kMaxTopK];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
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
        for (int c = w * 32 + lane; c < nv; c += WPT * 32) {
            const uint4 du = ldg_nc_v4(dy + t * H + c * 8);
            uint4 ou[kMaxTopK];
            if (d_w) {
#pragma unroll
                for (int j = 0; j < kMaxTopK; ++j)
                    ou[j] = pos[j] >= 0 ? ldg_nc_v4(o + int64_t(pos[j]) * H + c * 8) : make_uint4(0, 0, 0, 0);
            }
            float d[8];
            unpack8(du, d);
            if (d_w) {
#pragma unroll
                for (int j = 0; j < kMaxTopK; ++j) {
                    float x[8];
                    unpack8(ou[j], x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = fmaf(x[i], d[i], dot[j]);
                }
            }
            if (d_o) {
#pragma unroll
                for (int j = 0; j < kMaxTopK; ++j) {
                    if (pos[j] < 0) continue;
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = g[j] * d[i];
                    *reinterpret_cast<uint4*>(d_o + int64_t(pos[j]) * H + c * 8) = pack8(x);
                }
                if (ps >= 0) *reinterpret_cast<uint4*>(d_o + int64_t(ps) * H + c * 8) = du;
            }
        }
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
        for (int i = 0; i < WPT; ++i) s += part[tl * WPT + i][lane];
        d_w[t * k + lane] = s;
    }
}

cudaError_t launch_combine_backward(int T, int H, int k, int S, int R, const uint16_t* dy, const uint16_t* o,
                                    const int32_t* inv_pos, const float* gw, uint16_t* d_o, float* d_w, cudaStream_t st) {
    // as many warps as the row has 512-byte pieces (a lane then has a vector of its own), up to the CTA
    if (H <= 256)
        combine_backward_kernel<1><<<(T + 7) / 8, 256, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    else if (H <= 512)
        combine_backward_kernel<2><<<(T + 3) / 4, 256, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    else if (H <= 1024)
        combine_backward_kernel<4><<<(T + 1) / 2, 256, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    else
        combine_backward_kernel<8><<<T, 256, 0, st>>>(T, H, k, S, R, dy, o, inv_pos, gw, d_o, d_w);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ permutation
// One thread per 16-byte column of a token; the router's rows (fp32, two vectors per column) are
// small enough to come from L2.
template <bool ROUTER>
__global__ void __launch_bounds__(256) permute_backward_kernel(int T, int nv, int k, int S, int E, int R,
                                                               const uint16_t* __restrict__ dxs,
                                                               const int32_t* __restrict__ inv_pos,
                                                               const int32_t* __restrict__ idx,
                                                               const float* __restrict__ dl,
                                                               const float* __restrict__ wr, uint16_t* __restrict__ dx) {
    const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (at >= int64_t(T) * nv) return;
    const int t = int(at <= 0xFFFFFFFFll ? int64_t(uint32_t(at) / uint32_t(nv)) : at / nv);
    const int c = int(at - int64_t(t) * nv);
    uint4 u[kMaxTopK + 1];
#pragma unroll
    for (int j = 0; j < kMaxTopK + 1; ++j) {
        int p = -1;
        if (j < kMaxTopK) { if (j < k) p = inv_pos[int64_t(t) * k + j]; }
        else if (S) p = inv_pos[int64_t(T) * k + t];
        u[j] = p >= 0 && p < R ? ldg_nc_v4(dxs + (int64_t(p) * nv + c) * 8) : make_uint4(0, 0, 0, 0);
    }
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (ROUTER) {
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
            if (j >= k) break;
            const int e = idx[int64_t(t) * k + j];
            if (e < 0 || e >= E) continue;
            const float d = dl[int64_t(t) * k + j];
            const float4* w = reinterpret_cast<const float4*>(wr) + (int64_t(e) * nv + c) * 2;
            const float4 a = __ldg(w), b = __ldg(w + 1);
            acc[0] = fmaf(d, a.x, acc[0]); acc[1] = fmaf(d, a.y, acc[1]); acc[2] = fmaf(d, a.z, acc[2]); acc[3] = fmaf(d, a.w, acc[3]);
            acc[4] = fmaf(d, b.x, acc[4]); acc[5] = fmaf(d, b.y, acc[5]); acc[6] = fmaf(d, b.z, acc[6]); acc[7] = fmaf(d, b.w, acc[7]);
        }
    }
#pragma unroll
    for (int j = 0; j < kMaxTopK + 1; ++j) {
        float f[8];
        unpack8(u[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    *reinterpret_cast<uint4*>(dx + at * 8) = pack8(acc);
}

cudaError_t launch_permute_backward(int T, int H, int k, int S, int E, int R, const uint16_t* dxs, const int32_t* inv_pos,
                                    const int32_t* idx, const float* dl, const float* wr, uint16_t* dx, cudaStream_t st) {
    const int nv = H / 8;
    const int64_t blocks = (int64_t(T) * nv + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    if (wr) permute_backward_kernel<true><<<unsigned(blocks), 256, 0, st>>>(T, nv, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx);
    else permute_backward_kernel<false><<<unsigned(blocks), 256, 0, st>>>(T, nv, k, S, E, R, dxs, inv_pos, idx, dl, wr, dx);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ router
// The sorted order makes dWr a segmented sum over consecutive rows.  Segments are fixed runs of
// `seg` sorted rows; a CTA sums one segment for 1024 columns, expert by expert.  An expert that
// lies inside one segment is written directly; one that crosses a segment border leaves a partial
// sum per segment -- slot 2s (the rows at the segment's start) or 2s + 1 (the rows at its end) --
// and route_backward_join_kernel adds them in segment order.
constexpr int kRbThreads = 128;
constexpr int kRbCols = kRbThreads * 8;
constexpr int kRbMaxSeg = 64;

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
    float* part;     // [2 nseg, H]
    float* part_b;   // [2 nseg]
};

// gradient of the kept logit of flat pair p = t k + j
__device__ __forceinline__ float dlogit_of(const RouteBackward& a, int p) {
    const int t0 = p / a.k * a.k;
    float s = 0.f;
    for (int j = 0; j < a.k; ++j) s = fmaf(a.gw[t0 + j], a.dgw[t0 + j], s);
    return a.gw[p] * (a.dgw[p] - s);
}

__global__ void __launch_bounds__(kRbThreads) route_backward_kernel(RouteBackward a) {
    __shared__ float s_dl[kRbMaxSeg];
    __shared__ int s_tok[kRbMaxSeg];
    __shared__ int s_e[kRbMaxSeg];
    const int tid = threadIdx.x, sg = blockIdx.x;
    const int r0 = sg * a.seg;
    const int rows = max(0, min(a.offsets ? a.offsets[a.E] : 0, a.P));   // routed rows
    const int n = max(0, min(a.seg, rows - r0));
    if (blockIdx.y == 0 && tid < a.seg && r0 + tid < a.P) a.dlogits[r0 + tid] = dlogit_of(a, r0 + tid);
    if (!a.dw && !a.db) return;
    if (tid < n) {
        const int flat = a.sorted_flat[r0 + tid];
        const bool ok = flat >= 0 && flat < a.P;
        int e = ok ? a.idx[flat] : -1;
        if (e >= a.E) e = -1;
        s_e[tid] = e;
        s_tok[tid] = ok ? flat / a.k : 0;
        s_dl[tid] = ok ? dlogit_of(a, flat) : 0.f;
    }
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
            u[i] = in && b + i < n ? ldg_nc_v4(a.x + int64_t(s_tok[b + i]) * a.H + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = b + i;
            if (r >= n) break;
            const float d = s_dl[r];
            float f[8];
            unpack8(u[i], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] = fmaf(d, f[c], acc[c]);
            accb += d;
            const int e = s_e[r];
            if (r + 1 == n || s_e[r + 1] != e) {          // the run of this expert's rows ends here
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

// experts without rows get zeros; experts of several segments the sum of their partial sums
__global__ void __launch_bounds__(256) route_backward_join_kernel(RouteBackward a) {
    const int e = blockIdx.x;
    const int lo = a.offsets[e], hi = a.offsets[e + 1];
    const bool none = hi <= lo || lo < 0 || hi > a.P;
    const int s0 = none ? 0 : lo / a.seg, s1 = none ? 0 : (hi - 1) / a.seg;
    if (!none && s0 == s1) return;
    const int col = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int first = 2 * s0 + (lo % a.seg ? 1 : 0);
    if (a.dw && col < a.H) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!none) {
            s = *reinterpret_cast<const float4*>(a.part + int64_t(first) * a.H + col);
#pragma unroll 4
            for (int g = s0 + 1; g <= s1; ++g) {
                const float4 v = *reinterpret_cast<const float4*>(a.part + int64_t(2 * g) * a.H + col);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
        }
        *reinterpret_cast<float4*>(a.dw + int64_t(e) * a.H + col) = s;
    }
    if (a.db && blockIdx.y == 0 && threadIdx.x == 0) {
        float s = 0.f;
        if (!none) {
            s = a.part_b[first];
            for (int g = s0 + 1; g <= s1; ++g) s += a.part_b[2 * g];
        }
        a.db[e] = s;
    }
}

cudaError_t launch_route_backward(int T, int H, int k, int E, const uint16_t* x, const int32_t* idx, const float* gw,
                                  const float* dgw, const int32_t* offsets, const int32_t* sorted_flat, float* dlogits,
                                  float* dw, float* db, float* part, cudaStream_t st) {
    RouteBackward a{};
    a.T = T; a.H = H; a.k = k; a.E = E; a.P = T * k;
    // short segments until they fill the SMs, then longer ones (fewer partial sums)
    a.seg = a.P <= 16384 ? 16 : kRbMaxSeg;
    a.nseg = (a.P + a.seg - 1) / a.seg;
    a.x = x; a.idx = idx; a.gw = gw; a.dgw = dgw;
    a.offsets = offsets; a.sorted_flat = sorted_flat;
    a.dlogits = dlogits; a.dw = dw; a.db = db;
    a.part = part;
    a.part_b = part + int64_t(2) * a.nseg * H;
    const int cols = dw ? (H + kRbCols - 1) / kRbCols : 1;
    route_backward_kernel<<<dim3(a.nseg, cols), kRbThreads, 0, st>>>(a);
    if (dw || db) route_backward_join_kernel<<<dim3(E, dw ? (H + 1023) / 1024 : 1), 256, 0, st>>>(a);
    return cudaGetLastError();
}

size_t route_backward_part_bytes(int T, int H, int k) {
    const int P = T * k, seg = P <= 16384 ? 16 : kRbMaxSeg, nseg = (P + seg - 1) / seg;
    return nseg > 1 ? size_t(2) * nseg * (size_t(H) + 1) * sizeof(float) : 0;
}

}  // namespace ftmoe
