// mx4_quant.cu -- quantisation to the microscaled 4-bit format and back
// (OCP Microscaling Formats (MX) Specification v1.0, section 6.3), and a2's row copy in
// that format ("Llama 3 Meets MoE", section 3 "容量因子", for the dispatch itself).
//
// One thread per block of 32 columns.  Bound by memory: 2 bytes read and 0.53 written
// per bf16 element (and the reverse).
#include "mx4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load_block(const T *src, int n, float (&v)[32])
{
    constexpr int V = Vec<T>::N;
#pragma unroll
    for (int i = 0; i < 32; i += V) {
        if (i < n) {  // n is a multiple of 8
            const uint4 w = ld_nc(src + i);
            if constexpr (V == 8) {
                bf16x8_to_f32(w, &v[i]);
            } else {
                v[i] = __uint_as_float(w.x);
                v[i + 1] = __uint_as_float(w.y);
                v[i + 2] = __uint_as_float(w.z);
                v[i + 3] = __uint_as_float(w.w);
            }
        } else {
#pragma unroll
            for (int q = 0; q < V; ++q)
                v[i + q] = 0.f;
        }
    }
}

// codes of one block and its scale byte
__device__ __forceinline__ uint4 quantize_block(float (&v)[32], uint32_t &byte)
{
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
    byte = mx4_scale_byte(amax);
    if (byte == 255u)
        return make_uint4(0, 0, 0, 0);
    const float inv = mx4_inverse(byte);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = v[8 * j + i] * inv;
        c[j] = mx4_codes8(t);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// blocks of the padded matrix: tr * 128 rows, tk * 4 blocks (those outside are zero bytes)
template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_quantize_kernel(const T *__restrict__ src, int64_t G, int rows, int K, int64_t ld,
                        uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    pdl_wait();
    pdl_trigger();
    const int k32 = mx4_k32(K), tk = (K + 127) / 128, nb = tk * 4;
    const int64_t rp = (int64_t)(rows + 127) / 128 * 128, total = G * rp * nb;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        const int b = (int)(i % nb);
        const int64_t gr = i / nb, g = gr / rp;
        const int r = (int)(gr - g * rp);
        uint32_t byte = 0;
        if (r < rows && b * 32 < k32) {
            float v[32];
            load_block(src + (g * rows + r) * ld + b * 32, K - b * 32, v);
            const uint4 c = quantize_block(v, byte);
            st_v4(codes + (g * rows + r) * (k32 / 2) + b * 16, c);
        }
        scales[mx4_scale_at(g * (rp / 128), tk, r, b)] = (uint8_t)byte;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int64_t G, int rows, int K, int64_t ld, T *__restrict__ dst)
{
    pdl_wait();
    pdl_trigger();
    const int k32 = mx4_k32(K), tk = (K + 127) / 128, nb = k32 / 32;
    const int64_t tr = (rows + 127) / 128, total = G * rows * nb;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        const int b = (int)(i % nb);
        const int64_t gr = i / nb, g = gr / rows;
        const int r = (int)(gr - g * rows);
        const float sc = mx4_scale(scales[mx4_scale_at(g * tr, tk, r, b)]);
        const uint4 c = ld_nc(codes + gr * (k32 / 2) + b * 16);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        T *out = dst + gr * ld + b * 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (b * 32 + 8 * j >= K)
                break;
            uint32_t h[4];
            mx4_halves8(w[j], h);
            float v[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[q]));
                v[2 * q] = f.x * sc;
                v[2 * q + 1] = f.y * sc;
            }
            if constexpr (sizeof(T) == 2) {
                st_v4(out + 8 * j, f32x8_to_bf16(v));
            } else {
                float4 *o = reinterpret_cast<float4 *>(out + 8 * j);
                o[0] = make_float4(v[0], v[1], v[2], v[3]);
                o[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    }
}

// one thread per block of a token row: quantised once, written to every kept row
template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_dispatch_kernel(const T *__restrict__ x, int Tn, int d, int k, int E,
                        const int32_t *__restrict__ idx, const int32_t *__restrict__ slot,
                        const int32_t *__restrict__ offsets, uint8_t *__restrict__ xq,
                        uint8_t *__restrict__ xs)
{
    pdl_wait();
    pdl_trigger();
    const int tk = (d + 127) / 128, nb = tk * 4;
    const int64_t total = (int64_t)Tn * nb;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        const int b = (int)(i % nb), t = (int)(i / nb);
        uint32_t byte = 0;
        uint4 c = make_uint4(0, 0, 0, 0);
        if (b * 32 < d) {
            float v[32];
            load_block(x + (int64_t)t * d + b * 32, 32, v);
            c = quantize_block(v, byte);
        }
        for (int j = 0; j < k; ++j) {
            const int row = slot[(int64_t)t * k + j], e = idx[(int64_t)t * k + j];
            if (row < 0 || e < 0 || e >= E)
                continue;
            const int off = offsets[e];
            if (b * 32 < d)
                st_v4(xq + (int64_t)row * (d / 2) + b * 16, c);
            xs[mx4_scale_at(mx4_expert_tile(off, e), tk, row - off, b)] = (uint8_t)byte;
        }
    }
}

dim3 grid_for(int64_t threads)
{
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    return dim3((unsigned)(blocks < 148 * 64 ? (blocks > 0 ? blocks : 1) : 148 * 64));
}

}  // namespace

cudaError_t launch_mx4_quantize(const void *src, int dtype, int G, int rows, int K, int64_t ld,
                                void *codes, void *scales, cudaStream_t s)
{
    const int64_t n = (int64_t)G * ((rows + 127) / 128 * 128) * ((K + 127) / 128 * 4);
    count_launch();
    if (dtype == MOE_BF16)
        return launch_pdl(mx4_quantize_kernel<bf16>, grid_for(n), dim3(kThreads), 0, s,
                          (const bf16 *)src, (int64_t)G, rows, K, ld, (uint8_t *)codes,
                          (uint8_t *)scales);
    return launch_pdl(mx4_quantize_kernel<float>, grid_for(n), dim3(kThreads), 0, s,
                      (const float *)src, (int64_t)G, rows, K, ld, (uint8_t *)codes,
                      (uint8_t *)scales);
}

cudaError_t launch_mx4_dequantize(const void *codes, const void *scales, int dtype, int G,
                                  int rows, int K, int64_t ld, void *dst, cudaStream_t s)
{
    const int64_t n = (int64_t)G * rows * (mx4_k32(K) / 32);
    count_launch();
    if (dtype == MOE_BF16)
        return launch_pdl(mx4_dequantize_kernel<bf16>, grid_for(n), dim3(kThreads), 0, s,
                          (const uint8_t *)codes, (const uint8_t *)scales, (int64_t)G, rows, K,
                          ld, (bf16 *)dst);
    return launch_pdl(mx4_dequantize_kernel<float>, grid_for(n), dim3(kThreads), 0, s,
                      (const uint8_t *)codes, (const uint8_t *)scales, (int64_t)G, rows, K, ld,
                      (float *)dst);
}

cudaError_t launch_mx4_dispatch(const moe_params_t *p, const void *x, const int32_t *idx,
                                const int32_t *slot, const int32_t *offsets, void *xq, void *xs,
                                cudaStream_t s)
{
    const int64_t n = (int64_t)p->T * ((p->d + 127) / 128 * 4);
    count_launch();
    if (p->dtype == MOE_BF16)
        return launch_pdl(mx4_dispatch_kernel<bf16>, grid_for(n), dim3(kThreads), 0, s,
                          (const bf16 *)x, p->T, p->d, p->k, p->E, idx, slot, offsets,
                          (uint8_t *)xq, (uint8_t *)xs);
    return launch_pdl(mx4_dispatch_kernel<float>, grid_for(n), dim3(kThreads), 0, s,
                      (const float *)x, p->T, p->d, p->k, p->E, idx, slot, offsets,
                      (uint8_t *)xq, (uint8_t *)xs);
}

}  // namespace moe
