// Quantisation of matrices to MXFP4 and back.
//
// A dense (rows, cols) matrix with cols a multiple of 32 is a flat sequence
// of blocks, so both kernels run over units of 8 elements: a thread reads 16
// bytes of bf16 (32 of fp32), the four threads of a block find its largest
// magnitude with two shuffles, and a thread writes its 8 codes as one 32-bit
// word.  Bound by HBM: 2 or 4 bytes and 17/32 byte per element (16384 x 7168 in
// bf16, there and back, 595 MB: 102 to 104 us, 5.8 TB/s).
#include <cuda_fp16.h>
#include "internal.h"
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;              // units a thread has in flight

template <typename XT>
__device__ __forceinline__ void load8(const XT* p, float (&v)[8]);

template <>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// units: rows * cols / 8, a multiple of 4; the four threads of a block are
// neighbouring lanes of one warp, so a warp's shuffles stay within whole
// blocks even where the last warp is partly idle.
template <typename XT>
__global__ void __launch_bounds__(THREADS)
mxfp4_quantize_kernel(const XT* __restrict__ x, long long units, uint32_t* __restrict__ codes,
                      uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_allow_next();
    const long long base = static_cast<long long>(blockIdx.x) * (THREADS * UNROLL) + threadIdx.x;
    float v[UNROLL][8];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const long long i = base + u * THREADS;
        if (i < units) load8(x + 8 * i, v[u]);
        else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const long long i = base + u * THREADS;
        // as integers, magnitudes order like their values and a NaN is largest
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[u][j]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t b = mxfp4_scale_byte(m);
        const float inv = mxfp4_inv_scale(b == 255u ? 127u : b);
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = v[u][j] * inv;
        if (i < units) {
            codes[i] = b == 255u ? 0u : f32x8_to_e2m1x8(q);
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(b);
        }
    }
}

template <typename XT>
__global__ void __launch_bounds__(THREADS)
mxfp4_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long units,
                        XT* __restrict__ out) {
    pdl_wait();
    pdl_allow_next();
    const long long base = static_cast<long long>(blockIdx.x) * (THREADS * UNROLL) + threadIdx.x;
    uint32_t c[UNROLL], s[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const long long i = base + u * THREADS;
        c[u] = i < units ? __ldg(codes + i) : 0u;
        s[u] = i < units ? __ldg(scales + (i >> 2)) : 0u;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const long long i = base + u * THREADS;
        if (i >= units) break;
        const float sc = e8m0_value(s[u]);
        uint32_t h[4];
        e2m1x8_to_f16x2(c[u], h);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            v[2 * j] = f.x * sc;
            v[2 * j + 1] = f.y * sc;
        }
        store8(out + 8 * i, v);
    }
}

// A thread per word of the tiled scales: word w of row r of a tile of 128 rows
// lies at 16 (r mod 32) + 4 (r div 32) of the tile's w-th 512 bytes.
__global__ void __launch_bounds__(THREADS)
mxfp4_tile_scales_kernel(const uint32_t* __restrict__ scales, long long total, int rows, int words, int tiles,
                         uint32_t* __restrict__ out) {
    pdl_wait();
    pdl_allow_next();
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    if (i >= total) return;
    const int lane = static_cast<int>(i & 127);
    const long long block = i >> 7;                        // (matrix, tile, word)
    const int w = static_cast<int>(block % words);
    const long long t = block / words;
    const int row = static_cast<int>(t % tiles) * 128 + (lane >> 2) + 32 * (lane & 3);
    // rows past the end: 2^0
    out[i] = row < rows ? __ldg(scales + (t / tiles * rows + row) * words + w) : 0x7F7F7F7Fu;
}

}  // namespace

cudaError_t launch_mxfp4_tile_scales(const uint8_t* scales, long long n_mats, int rows, int cols, uint8_t* tiled,
                                     cudaStream_t st) {
    const int words = cols / 128, tiles = (rows + 127) / 128;
    const long long total = n_mats * tiles * words * 128;
    const dim3 grid(static_cast<unsigned>((total + THREADS - 1) / THREADS));
    return launch_pdl(mxfp4_tile_scales_kernel, grid, dim3(THREADS), 0, st, 1, reinterpret_cast<const uint32_t*>(scales),
                      total, rows, words, tiles, reinterpret_cast<uint32_t*>(tiled));
}

cudaError_t launch_mxfp4_quantize(const void* x, int dtype, long long elems, uint8_t* codes, uint8_t* scales,
                                  cudaStream_t st) {
    const long long units = elems / 8;
    const long long blocks = (units + THREADS * UNROLL - 1) / (THREADS * UNROLL);
    const dim3 grid(static_cast<unsigned>(blocks)), block(THREADS);
    uint32_t* c = reinterpret_cast<uint32_t*>(codes);
    if (dtype == MOE_F32)
        return launch_pdl(mxfp4_quantize_kernel<float>, grid, block, 0, st, 1, static_cast<const float*>(x), units, c,
                          scales);
    return launch_pdl(mxfp4_quantize_kernel<__nv_bfloat16>, grid, block, 0, st, 1,
                      static_cast<const __nv_bfloat16*>(x), units, c, scales);
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, long long elems, void* out,
                                    int dtype, cudaStream_t st) {
    const long long units = elems / 8;
    const long long blocks = (units + THREADS * UNROLL - 1) / (THREADS * UNROLL);
    const dim3 grid(static_cast<unsigned>(blocks)), block(THREADS);
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
    if (dtype == MOE_F32)
        return launch_pdl(mxfp4_dequantize_kernel<float>, grid, block, 0, st, 1, c, scales, units,
                          static_cast<float*>(out));
    return launch_pdl(mxfp4_dequantize_kernel<__nv_bfloat16>, grid, block, 0, st, 1, c, scales, units,
                      static_cast<__nv_bfloat16*>(out));
}

}  // namespace moe
