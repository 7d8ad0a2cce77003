// MXFP4 quantisation of rows (weights from a checkpoint, activations), and of a batch's tokens
// straight into their expert-sorted places.  The format and the rounding are in mx4.cuh.
//
// One pass, bound by memory: a thread takes eight consecutive elements (one or two 16-byte loads),
// four neighbouring lanes share a 32-element block and exchange its maximum with two shuffles;
// kIlp vectors per thread are loaded before the first is used.
#include "decode_common.cuh"
#include "mx4.cuh"

namespace ftmoe {

constexpr int kQThreads = 256;
constexpr int kIlp = 4;

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr int kVecs = 1;
    static __device__ void unpack(const uint4 (&u)[1], float (&v)[8]) {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[2 * i] = bf16lo(w[i]); v[2 * i + 1] = bf16hi(w[i]); }
    }
    static __device__ void pack(const float (&v)[8], uint4 (&u)[1]) {
        u[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    static __device__ float scalar(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <> struct Elem<__half> {
    static constexpr int kVecs = 1;
    static __device__ void unpack(const uint4 (&u)[1], float (&v)[8]) {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
            v[2 * i] = __low2float(h);
            v[2 * i + 1] = __high2float(h);
        }
    }
    static __device__ void pack(const float (&v)[8], uint4 (&u)[1]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        u[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ float scalar(const __half* p) { return __half2float(*p); }
};
template <> struct Elem<float> {
    static constexpr int kVecs = 2;
    static __device__ void unpack(const uint4 (&u)[2], float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(u[i].x); v[4 * i + 1] = __uint_as_float(u[i].y);
            v[4 * i + 2] = __uint_as_float(u[i].z); v[4 * i + 3] = __uint_as_float(u[i].w);
        }
    }
    static __device__ void pack(const float (&v)[8], uint4 (&u)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            u[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                              __float_as_uint(v[4 * i + 3]));
    }
    static __device__ float scalar(const float* p) { return *p; }
};

// this lane's eight elements of a block shared by four neighbouring lanes -> codes and the scale byte
__device__ __forceinline__ uint32_t mx4_quad(const float (&v)[8], uint32_t& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    float mul;
    scale = mx4_scale_of(m, mul);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = v[i] * mul;
    const uint32_t c = e2m1x8(s);
    return scale == 255u ? 0u : c;
}

// nv = vectors of eight per row; total = rows * nv (a multiple of 4, so the four lanes of a block
// are in range together).  ALIGNED: rows start on 16-byte boundaries; otherwise element loads.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kQThreads) mx4_quantize_kernel(int64_t total, int nv, const T* __restrict__ x,
                                                                 int64_t stride, uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales, T* __restrict__ values) {
    constexpr int kV = Elem<T>::kVecs;
    const int64_t base = int64_t(blockIdx.x) * (kQThreads * kIlp) + threadIdx.x;
    float v[kIlp][8];
    uint4 u[kIlp][kV];
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
        const int64_t at = base + i * kQThreads;
        const int64_t id = at < total ? at : 0;
        // 32-bit division where it can be: a 64-bit one costs as much as the rest of the vector
        const int64_t row = id <= 0xFFFFFFFFll ? int64_t(uint32_t(id) / uint32_t(nv)) : id / nv;
        const T* p = x + row * stride + (id - row * nv) * 8;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int j = 0; j < kV; ++j) u[i][j] = ldg_nc_v4(reinterpret_cast<const uint4*>(p) + j);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = Elem<T>::scalar(p + j);
        }
    }
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
        const int64_t at = base + i * kQThreads;
        if constexpr (ALIGNED) Elem<T>::unpack(u[i], v[i]);
        uint32_t s;
        const uint32_t c = mx4_quad(v[i], s);
        if (at < total) {
            codes[at] = c;
            if ((at & 3) == 0) scales[at >> 2] = uint8_t(s);
            if (values) {
                float o[8];
                e2m1x8_values(c, e8m0_float(s), o);
                uint4 w[kV];
                Elem<T>::pack(o, w);
#pragma unroll
                for (int j = 0; j < kV; ++j) reinterpret_cast<uint4*>(values + at * 8)[j] = w[j];
            }
        }
    }
}

template <typename T>
static cudaError_t quantize_t(int64_t rows, int cols, const void* x, int64_t stride, uint8_t* codes, uint8_t* scales,
                              void* values, cudaStream_t st) {
    const int nv = cols / 8;
    const int64_t total = rows * nv;
    const int64_t blocks = (total + kQThreads * kIlp - 1) / (kQThreads * kIlp);
    const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (stride * int64_t(sizeof(T))) % 16 == 0;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    if (aligned)
        mx4_quantize_kernel<T, true><<<unsigned(blocks), kQThreads, 0, st>>>(
            total, nv, static_cast<const T*>(x), stride, reinterpret_cast<uint32_t*>(codes), scales, static_cast<T*>(values));
    else
        mx4_quantize_kernel<T, false><<<unsigned(blocks), kQThreads, 0, st>>>(
            total, nv, static_cast<const T*>(x), stride, reinterpret_cast<uint32_t*>(codes), scales, static_cast<T*>(values));
    return cudaGetLastError();
}

cudaError_t launch_mx4_quantize(int64_t rows, int cols, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                                uint8_t* scales, void* values, cudaStream_t st) {
    switch (dtype) {
        case FT_T_BF16: return quantize_t<__nv_bfloat16>(rows, cols, x, x_stride, codes, scales, values, st);
        case FT_T_FP16: return quantize_t<__half>(rows, cols, x, x_stride, codes, scales, values, st);
        default: return quantize_t<float>(rows, cols, x, x_stride, codes, scales, values, st);
    }
}

// Tokens into sorted order: each row of x is read and quantised once and its codes are written to
// the k (+ 1 shared) sorted places of the token's pairs, so a batch costs one read of x and R rows
// of 17/32 bytes per element written (a gather of bf16 rows writes 2 bytes per element).  A thread
// takes a whole 32-element block, so a place costs one 16-byte store and the scale byte (with eight
// elements per thread, four 4-byte stores: 2049 x 2816, nine places, 13.4 -> 8.4 us).
// A position outside [0, R) (a dropped pair) is skipped.
__global__ void __launch_bounds__(kQThreads) mx4_sorted_tokens_kernel(int T, int nb, int k, int S,
                                                                      const uint16_t* __restrict__ x,
                                                                      const int32_t* __restrict__ inv_pos,
                                                                      uint4* __restrict__ codes,
                                                                      uint8_t* __restrict__ scales) {
    const int R = T * k + S * T;
    const int64_t total = int64_t(T) * nb;
    const int64_t at = int64_t(blockIdx.x) * kQThreads + threadIdx.x;
    pdl_wait();
    pdl_trigger();      // after the wait: the permutation is final for the product that follows
    if (at >= total) return;
    const int t = int(at <= 0xFFFFFFFFll ? int64_t(uint32_t(at) / uint32_t(nb)) : at / nb);
    const int c = int(at - int64_t(t) * nb);
    uint4 u[4][1];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i][0] = ldg_nc_v4(reinterpret_cast<const uint4*>(x) + at * 4 + i);
    int pos[kMaxTopK + 1];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) pos[j] = j < k ? inv_pos[int64_t(t) * k + j] : -1;
    pos[kMaxTopK] = S ? inv_pos[int64_t(T) * k + t] : -1;
    float v[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Elem<__nv_bfloat16>::unpack(u[i], v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    }
    float mul;
    const uint32_t s = mx4_scale_of(m, mul);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= mul;
        q[i] = s == 255u ? 0u : e2m1x8(v[i]);
    }
#pragma unroll
    for (int j = 0; j < kMaxTopK + 1; ++j) {
        if (pos[j] < 0 || pos[j] >= R) continue;
        codes[size_t(pos[j]) * nb + c] = make_uint4(q[0], q[1], q[2], q[3]);
        scales[size_t(pos[j]) * nb + c] = uint8_t(s);
    }
}

cudaError_t launch_mx4_sorted_tokens(int T, int H, int k, int S, const uint16_t* x, const int32_t* inv_pos,
                                     uint8_t* codes, uint8_t* scales, cudaStream_t st) {
    if (T <= 0) return cudaSuccess;
    const int nb = H / 32;
    const int64_t blocks = (int64_t(T) * nb + kQThreads - 1) / kQThreads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mx4_sorted_tokens_kernel, T, nb, k, S, x, inv_pos, reinterpret_cast<uint4*>(codes), scales);
}

}  // namespace ftmoe
