// mx4_quant.cu -- quantisation to the microscaled 4-bit format and back
// (OCP Microscaling Formats (MX) Specification v1.0, section 6.3), and a2's row copy in
// that format ("Llama 3 Meets MoE", section 3 "容量因子", for the dispatch itself).
//
// Bound by memory: 2 bytes read and 0.53 written per bf16 element, and the reverse.  A lane
// holds 8 consecutive columns (16 bytes of bf16), so every load and store of a warp is a run
// of whole sectors; the 4 lanes of a block find its maximum in two shuffles, and the 16 lanes
// of 128 columns put the 4 scale bytes of a row together.  In the matrix kernels a warp takes
// 128 columns of 8 rows, the two neighbouring ones and those 32, 64 and 96 below, whose scale
// words are the 32 bytes of one sector of the tile; the loads of all 8 rows are in flight
// together.  The dispatch gives a thread a whole block (64 bytes of bf16 read, 16 of codes
// written to each row): with a row written twice its 16-byte stores count more than its loads
// (38.5 us against 47 with 8 columns a lane at T = 16384, d = 4096, top-2; 5.3 TB/s of the
// bytes in and out).  Quantising 8 x 2752 x 4096 bf16 takes 46 us (5.0 TB/s), the reverse 36
// (6.3 TB/s); 8 x 4096 x 1376 26 and 20 us (4.4 and 5.7 TB/s).
#include "mx4.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// 16 bytes read once.  Volatile: the loads of a unit are issued together, before the first is
// used.
__device__ __forceinline__ uint4 ld_now(const void *p)
{
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

template <typename T> struct Raw;  // 8 values as loaded
template <> struct Raw<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16 *p) { a = ld_now(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const { bf16x8_to_f32(a, v); }
};
template <> struct Raw<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = ld_now(p);
        b = ld_now(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float(w[i]);
    }
};

// The 8 codes of this lane and the scale byte of its block (4 neighbouring lanes).
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const Raw<T> &raw, uint32_t &byte)
{
    float v[8];
    raw.get(v);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    byte = mx4_scale_byte(amax);
    const float inv = mx4_inverse(byte == 255u ? 0u : byte);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] *= inv;
    const uint32_t c = mx4_codes8(v);
    return byte == 255u ? 0u : c;
}

// The scale word of this lane's row from the bytes of its 16 lanes (4 per block).
__device__ __forceinline__ uint32_t scale_word(uint32_t byte)
{
    uint32_t w = byte << (((threadIdx.x >> 2) & 3) * 8);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    return w;
}

// A warp's unit of a matrix (blockIdx.y, + gridDim.y, ...): TILES tile columns from kb on of
// rows 2 p + {0, 1} + 32 i of tile row tr.  Quantising takes 4, the next one's loads in flight
// while one is worked on (8 x 2752 x 4096 bf16: 46 us, 49 with 1); the reverse waits on little
// and takes 1 (36 us, 38 with 4).
constexpr int kQuantTiles = 4, kDequantTiles = 1;
struct Unit {
    int tr, p, kb;
    bool on;
};
template <int TILES>
__device__ __forceinline__ Unit unit_at(int trs, int tk)
{
    const uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint32_t per = (uint32_t)(tk + TILES - 1) / TILES;
    const uint32_t r = u / per;
    Unit o;
    o.kb = (int)(u - r * per) * TILES;
    o.p = (int)(r & 15u);
    o.tr = (int)(r >> 4);
    o.on = o.tr < trs;
    return o;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_quantize_kernel(const T *__restrict__ src, int G, int rows, int K, int64_t ld,
                        uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    pdl_wait();
    pdl_trigger();
    const int k32 = mx4_k32(K), tk = (K + 127) / 128, trs = (rows + 127) / 128;
    const Unit at = unit_at<kQuantTiles>(trs, tk);
    if (!at.on)
        return;
    const int l = threadIdx.x & 15, r0 = 2 * at.p + ((threadIdx.x >> 4) & 1);
    const int row0 = at.tr * 128 + r0, col = at.kb * 128 + 8 * l;
    for (int64_t g = blockIdx.y; g < G; g += gridDim.y) {
        const T *sp = src + (g * rows + row0) * ld + col;
        Raw<T> next[4];
        auto load = [&](int j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (row0 + 32 * i < rows && col + 128 * j < K)  // K is a multiple of 8
                    next[i].load(sp + 32 * i * ld + 128 * j);
                else
                    next[i].zero();
            }
        };
        load(0);
#pragma unroll 1
        for (int j = 0; j < kQuantTiles && at.kb + j < tk; ++j) {
            Raw<T> raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[i] = next[i];
            if (j + 1 < kQuantTiles)
                load(j + 1);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t byte;
                const uint32_t c = quantize8(raw[i], byte);
                if (row0 + 32 * i < rows && col + 128 * j < k32)
                    *reinterpret_cast<uint32_t *>(codes + (g * rows + row0 + 32 * i) * (k32 / 2) +
                                                  (col + 128 * j) / 2) = c;
                w[i] = scale_word(byte);
            }
            if (l == 0)
                st_v4(scales + ((g * trs + at.tr) * tk + at.kb + j) * kMx4Tile + r0 * 16,
                      make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                          int G, int rows, int K, int64_t ld, T *__restrict__ dst)
{
    pdl_wait();
    pdl_trigger();
    const int k32 = mx4_k32(K), tk = (K + 127) / 128, trs = (rows + 127) / 128;
    const Unit at = unit_at<kDequantTiles>(trs, tk);
    if (!at.on)
        return;
    const int l = threadIdx.x & 15, r0 = 2 * at.p + ((threadIdx.x >> 4) & 1);
    const int row0 = at.tr * 128 + r0, col = at.kb * 128 + 8 * l;
    for (int64_t g = blockIdx.y; g < G; g += gridDim.y) {
        uint4 words[kDequantTiles];
        uint32_t c[kDequantTiles][4];
#pragma unroll
        for (int j = 0; j < kDequantTiles; ++j) {
            words[j] = make_uint4(0, 0, 0, 0);
            if (at.kb + j < tk)
                words[j] = ld_nc_na(scales + ((g * trs + at.tr) * tk + at.kb + j) * kMx4Tile + r0 * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[j][i] = row0 + 32 * i < rows && col + 128 * j < K
                              ? __ldg(reinterpret_cast<const uint32_t *>(
                                    codes + (g * rows + row0 + 32 * i) * (k32 / 2) + (col + 128 * j) / 2))
                              : 0u;
        }
#pragma unroll
        for (int j = 0; j < kDequantTiles; ++j) {
            const uint32_t w[4] = {words[j].x, words[j].y, words[j].z, words[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sc = mx4_scale((w[i] >> ((l >> 2) * 8)) & 255u);
                uint32_t h[4];
                mx4_halves8(c[j][i], h);
                float v[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[q]));
                    v[2 * q] = f.x * sc;
                    v[2 * q + 1] = f.y * sc;
                }
                if (row0 + 32 * i < rows && col + 128 * j < K) {
                    T *out = dst + (g * rows + row0 + 32 * i) * ld + col + 128 * j;
                    if constexpr (sizeof(T) == 2) {
                        st_v4(out, f32x8_to_bf16(v));
                    } else {
                        float4 *o = reinterpret_cast<float4 *>(out);
                        o[0] = make_float4(v[0], v[1], v[2], v[3]);
                        o[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void load_block(const T *src, float (&v)[32])
{
    constexpr int V = Vec<T>::N;
#pragma unroll
    for (int i = 0; i < 32; i += V) {
        const uint4 w = ld_nc(src + i);
        if constexpr (V == 8) {
            bf16x8_to_f32(w, &v[i]);
        } else {
            v[i] = __uint_as_float(w.x);
            v[i + 1] = __uint_as_float(w.y);
            v[i + 2] = __uint_as_float(w.z);
            v[i + 3] = __uint_as_float(w.w);
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
            load_block(x + (int64_t)t * d + b * 32, v);
            c = quantize_block(v, byte);
        }
        for (int j = 0; j < k; ++j) {
            const int row = slot[(int64_t)t * k + j], e = idx[(int64_t)t * k + j];
            if (row < 0 || e < 0 || e >= E)
                continue;
            const int off = offsets[e];
            if (row >= Tn * k || off < 0 || off > row)
                continue;  // no dispatch writes such tables; the buffers end here
            if (b * 32 < d)
                st_v4(xq + (int64_t)row * (d / 2) + b * 16, c);
            xs[mx4_scale_at(mx4_expert_tile(off, e), tk, row - off, b)] = (uint8_t)byte;
        }
    }
}

// CTAs of a matrix batch: units of a matrix x matrices; false if a matrix has too many
bool matrix_grid(int G, int64_t rows, int64_t K, int tiles, dim3 *grid)
{
    const int64_t tk = (K + 127) / 128;
    const int64_t units = (rows + 127) / 128 * 16 * ((tk + tiles - 1) / tiles);
    const int64_t blocks = (units + kWarps - 1) / kWarps;
    *grid = dim3((unsigned)blocks, (unsigned)(G < 65535 ? G : 65535));
    return blocks < ((int64_t)1 << 31) / kWarps;
}

}  // namespace

cudaError_t launch_mx4_quantize(const void *src, int dtype, int G, int rows, int K, int64_t ld,
                                void *codes, void *scales, cudaStream_t s)
{
    dim3 grid;
    if (!matrix_grid(G, rows, K, kQuantTiles, &grid))
        return cudaErrorInvalidConfiguration;
    count_launch();
    if (dtype == MOE_BF16)
        return launch_pdl(mx4_quantize_kernel<bf16>, grid, dim3(kThreads), 0, s, (const bf16 *)src,
                          G, rows, K, ld, (uint8_t *)codes, (uint8_t *)scales);
    return launch_pdl(mx4_quantize_kernel<float>, grid, dim3(kThreads), 0, s, (const float *)src,
                      G, rows, K, ld, (uint8_t *)codes, (uint8_t *)scales);
}

cudaError_t launch_mx4_dequantize(const void *codes, const void *scales, int dtype, int G,
                                  int rows, int K, int64_t ld, void *dst, cudaStream_t s)
{
    dim3 grid;
    if (!matrix_grid(G, rows, K, kDequantTiles, &grid))
        return cudaErrorInvalidConfiguration;
    count_launch();
    if (dtype == MOE_BF16)
        return launch_pdl(mx4_dequantize_kernel<bf16>, grid, dim3(kThreads), 0, s,
                          (const uint8_t *)codes, (const uint8_t *)scales, G, rows, K, ld,
                          (bf16 *)dst);
    return launch_pdl(mx4_dequantize_kernel<float>, grid, dim3(kThreads), 0, s,
                      (const uint8_t *)codes, (const uint8_t *)scales, G, rows, K, ld,
                      (float *)dst);
}

cudaError_t launch_mx4_dispatch(const moe_params_t *p, const void *x, const int32_t *idx,
                                const int32_t *slot, const int32_t *offsets, void *xq, void *xs,
                                cudaStream_t s)
{
    const int64_t n = (int64_t)p->T * ((p->d + 127) / 128 * 4), blocks = (n + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(blocks < 148 * 64 ? blocks : 148 * 64));
    count_launch();
    if (p->dtype == MOE_BF16)
        return launch_pdl(mx4_dispatch_kernel<bf16>, grid, dim3(kThreads), 0, s, (const bf16 *)x,
                          p->T, p->d, p->k, p->E, idx, slot, offsets, (uint8_t *)xq, (uint8_t *)xs);
    return launch_pdl(mx4_dispatch_kernel<float>, grid, dim3(kThreads), 0, s, (const float *)x,
                      p->T, p->d, p->k, p->E, idx, slot, offsets, (uint8_t *)xq, (uint8_t *)xs);
}

}  // namespace moe
