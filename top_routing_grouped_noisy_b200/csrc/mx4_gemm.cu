// mx4_gemm.cu -- a3/a4 with both operands microscaled 4-bit ("LLaMA-MoE v2", code sample
// "代码实现示例", class Expert, on MXFP4 values): a persistent grouped GEMM on the
// block-scaled tensor-core products (tcgen05.mma kind::mxf4, f32 accumulators in TMEM).
//
//   a3: h = silu(xq W1_e^T) * (xq W3_e^T), quantised in the epilogue to h_q / h_s
//   a4: out = hq W2_e^T, rounded to bf16
//
// Operands.  Codes are K-major, two per byte, so a 128-byte swizzled row holds 256
// columns and one tcgen05.mma (K = 64) takes 32 bytes of it: byte for byte the walk of
// the bf16 GEMM with four times the columns.  Scales travel in their 512-byte tiles
// (128 rows x 4 blocks of 32 columns): one untiled bulk copy per operand and row tile
// brings a stage's tiles, and tcgen05.cp (32x128b, to all four lane quarters) moves them
// to TMEM, 4 columns per tile; a product takes the 2-byte half of its column's words
// that the scale ids in its instruction descriptor name.  tcgen05.cp and tcgen05.mma of
// one thread run in issue order, so the copies need no wait of their own.
//
// Work: tiles of 128 rows x BN columns over every expert, listed on the device from the
// offsets.  TMEM: two accumulators of BN columns, then the scale columns (24 per set,
// four sets).  Roles as in the bf16 kernel: warp 0 TMA producer, warp 1 TMEM allocator
// and issuer, warps 2-9 epilogue (each thread one row, half of the columns).
//
// Every mbarrier wait is bounded: past the limit the kernel records
// MOE_ERR_DEVICE_TIMEOUT, stops every role, drains its copies and products (bounded
// again) and frees TMEM.  No TMA load here uses cluster multicast.
#include <mutex>

#include "mx4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace mxg {

using namespace tc;

constexpr int BM = 128;
constexpr int BKB = 128;            // bytes of a stage row: 256 columns
constexpr int BKC = 256;            // columns of a stage
constexpr int ACC = 2;
constexpr int kSfSets = 4;          // scale column sets in TMEM
constexpr int kSfCols = 24;         // per set: 2 x (4 A + 8 B)
constexpr int TMEM_COLS = 512;
constexpr int NUM_THREADS = 320;
constexpr int EPI_WARPS = 8;
constexpr int kMaxStages = 8;

enum { EPI_UP = 0, EPI_DOWN = 1 };

struct Aux {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tfull[ACC];
    uint64_t tempty[ACC];
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t off[MOE_MAX_EXPERTS + 1];
    int32_t tstart[MOE_MAX_EXPERTS + 1];
};

template <int BN>
struct Geo {
    static constexpr int BT = (BN + 127) / 128;             // B scale tiles of a tile
    static constexpr int A_BYTES = BM * BKB;
    static constexpr int B_BYTES = BN * BKB;
    static constexpr int SFA = 2 * kMx4Tile;                // two K tiles per stage
    static constexpr int SFB = BT * 2 * kMx4Tile;
    static constexpr int STAGE = A_BYTES + B_BYTES + SFA + SFB;
    static constexpr int FIXED = 1024 + (int)sizeof(Aux);
    static constexpr int FIT = (227 * 1024 - FIXED) / STAGE;
    static constexpr int STAGES = FIT < kMaxStages ? FIT : kMaxStages;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static constexpr int SF_COL = ACC * BN;
    // kind::mxf4, A and B e2m1 K-major, e8m0 scales, M = 128
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                      (1u << 23) | ((uint32_t)(BM >> 7) << 27);
    static_assert(BN % 64 == 0 && STAGE % 1024 == 0, "tile");
    static_assert(SF_COL + kSfSets * kSfCols <= TMEM_COLS, "TMEM columns");
    static_assert(SMEM > 114 * 1024, "one CTA per SM: TMEM is allocated before the grid wait");
};

// smem descriptor of a scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups 128 B apart
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

__device__ __forceinline__ void sf_copy(uint32_t tmem, uint32_t saddr)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sf_desc(saddr))
                 : "memory");
}

__device__ __forceinline__ void umma_mx4(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

struct Tile {
    int e, row0, row_end, n0, off;
};

template <int BN>
__device__ __forceinline__ Tile decode_tile(const Aux *aux, int tile)
{
    Tile t;
    int e = 0;
    while (tile >= aux->tstart[e + 1])
        ++e;
    const int local = tile - aux->tstart[e];
    const int rows = aux->off[e + 1] - aux->off[e];
    const int mtiles = (rows + BM - 1) / BM;
    t.e = e;
    t.off = aux->off[e];
    t.row0 = t.off + (local % mtiles) * BM;
    t.row_end = aux->off[e + 1];
    t.n0 = (local / mtiles) * BN;
    return t;
}

struct GemmArgs {
    const uint8_t *a_s;        // scales of the rows
    const uint8_t *b_s;        // scales of the experts
    const int32_t *offsets;
    void *out;                 // DOWN: bf16 [rows][ld]; UP: h codes [rows][h32/2]
    uint8_t *h_s;              // UP: scales of h
    int E, N, K32;             // N: rows of an expert's matrix
    int n_valid;               // UP: neurons m; DOWN: columns d
    int ld;                    // DOWN: d; UP: h32 / 2
    int32_t *status;
    uint64_t wait_ns;
};

// 32 accumulator columns c..c+31 of this thread's row: 16 gate and 16 up values
__device__ __forceinline__ void swiglu16(const uint32_t (&v)[32], float *h)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float g = __uint_as_float(v[i]), u = __uint_as_float(v[16 + i]);
        // approximate division (2 ulp; 0 once 1 + e^-g > 2^126, silu's limit), far below
        // the 4-bit rounding that follows
        h[i] = __fdividef(g, 1.0f + __expf(-g)) * u;
    }
}

template <int EPI, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ GemmArgs a)
{
    using G = Geo<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Aux *aux = reinterpret_cast<Aux *>(smem + G::STAGES * G::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int32_t *abort_flag = &aux->abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::STAGES; ++s) {
            mbar_init(smem_u32(&aux->full[s]), 1);
            mbar_init(smem_u32(&aux->empty[s]), 1);
        }
        for (int i = 0; i < ACC; ++i) {
            mbar_init(smem_u32(&aux->tfull[i]), 1);
            mbar_init(smem_u32(&aux->tempty[i]), EPI_WARPS);
        }
        mbar_init(smem_u32(&aux->drain), 1);
        aux->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&aux->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();
    const int n_tiles = (a.N + BN - 1) / BN;
    if (warp == 2) {
        for (int i = lane; i <= a.E; i += 32)
            aux->off[i] = a.offsets[i];
        __syncwarp();
        if (lane == 0) {
            int acc = 0;
            for (int e = 0; e < a.E; ++e) {
                aux->tstart[e] = acc;
                acc += (aux->off[e + 1] - aux->off[e] + BM - 1) / BM * n_tiles;
            }
            aux->tstart[a.E] = acc;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = aux->tmem_base;
    const int total = aux->tstart[a.E];
    const int num_kb = (a.K32 + BKC - 1) / BKC;
    const int tk = (a.K32 + 127) / 128;          // K tiles of a scale tile row
    const int trb = (a.N + 127) / 128;           // scale tile rows of an expert's matrix
    const uint32_t smem_base = smem_u32(smem);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            int64_t fills = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                const Tile t = decode_tile<BN>(aux, tile);
                const uint8_t *sa_src =
                    a.a_s + (mx4_expert_tile(t.off, t.e) + (t.row0 - t.off) / BM) * tk * kMx4Tile;
                const int nb0 = t.n0 / 128;
                const int nbt = min(G::BT, trb - nb0);  // B scale tiles that exist
                const uint8_t *sb_src = a.b_s + ((int64_t)t.e * trb + nb0) * tk * kMx4Tile;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&aux->empty[stage]), phase ^ 1u, a.wait_ns, abort_flag,
                                   a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&aux->full[stage]);
                    const uint32_t sa = smem_base + stage * G::STAGE, sb = sa + G::A_BYTES;
                    const uint32_t sfa = sb + G::B_BYTES, sfb = sfa + G::SFA;
                    const uint32_t kt = (uint32_t)min(2, tk - 2 * kb) * kMx4Tile;
                    mbar_expect_tx(fb, (uint32_t)(G::A_BYTES + G::B_BYTES) + kt * (1 + nbt));
                    tma_load_2d(&tmA, fb, sa, kb * (BKB / 2), t.row0);
                    tma_load_3d(&tmB, fb, sb, kb * (BKB / 2), t.n0, t.e);
                    bulk_load(sfa, sa_src + (int64_t)2 * kb * kMx4Tile, kt, fb);
                    for (int i = 0; i < nbt; ++i)
                        bulk_load(sfb + i * 2 * kMx4Tile,
                                  sb_src + ((int64_t)i * tk + 2 * kb) * kMx4Tile, kt, fb);
                    ++fills;
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < G::STAGES; ++s) {
                const int64_t n = fills / G::STAGES + (s < fills % G::STAGES ? 1 : 0);
                if (n > 0)
                    mbar_drain(smem_u32(&aux->full[s]), (uint32_t)((n - 1) & 1));
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------------------------------------------------- issuer
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0, set = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            const int nk = (a.K32 + 63) / 64;  // products along K
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                const Tile t = decode_tile<BN>(aux, tile);
                // first B scale column inside the copied tiles: one column per 32 rows
                const uint32_t b_shift = (uint32_t)(t.n0 % 128 / 32);
                if (!mbar_wait(smem_u32(&aux->tempty[acc]), acc_phase ^ 1u, a.wait_ns, abort_flag,
                               a.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&aux->full[stage]), phase, a.wait_ns, abort_flag,
                                   a.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_base + stage * G::STAGE, sb = sa + G::A_BYTES;
                    const uint32_t sfa = sb + G::B_BYTES, sfb = sfa + G::SFA;
                    const uint32_t sf = tmem_base + (uint32_t)(G::SF_COL + set * kSfCols);
                    const int halves = min(2, tk - 2 * kb);
                    for (int hh = 0; hh < halves; ++hh) {
                        sf_copy(sf + hh * 12, sfa + hh * kMx4Tile);
#pragma unroll
                        for (int i = 0; i < G::BT; ++i)
                            sf_copy(sf + hh * 12 + 4 + i * 4, sfb + (i * 2 + hh) * kMx4Tile);
                    }
                    const uint64_t da = sdesc(sa), db = sdesc(sb);
                    const int ks = min(4, nk - 4 * kb);
                    for (int k = 0; k < ks; ++k) {
                        const uint32_t id = (uint32_t)(k & 1) * 2u;
                        const uint32_t col = sf + (uint32_t)(k >> 1) * 12;
                        umma_mx4(d_tmem, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k),
                                 G::IDESC | (id << 4) | (id << 29), col, col + 4 + b_shift,
                                 (kb | k) != 0);
                    }
                    umma_commit(smem_u32(&aux->empty[stage]));
                    set = (set + 1) % kSfSets;
                    if (++stage == G::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                umma_commit(smem_u32(&aux->tfull[acc]));
                if (++acc == ACC) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            umma_commit(smem_u32(&aux->drain));
            mbar_drain(smem_u32(&aux->drain), 0);
        }
    } else {
        // -------------------------------------------------------------- epilogue
        const int lane_base = (warp & 3) * 32;
        const bool upper = (warp - 2) / 4 != 0;
        // 64-column groups of the tile: the first half of the warps takes the larger half
        constexpr int kGroups = BN / 64, kHalf0 = (kGroups + 1) / 2;
        const int g_first = upper ? kHalf0 : 0, g_end = upper ? kGroups : kHalf0;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
            const Tile t = decode_tile<BN>(aux, tile);
            if (!mbar_wait(smem_u32(&aux->tfull[acc]), acc_phase, a.wait_ns, abort_flag, a.status))
                break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)lane_base << 16) + (uint32_t)(acc * BN);
            const int row = t.row0 + lane_base + lane;
            const bool rv = row < t.row_end;
            if (t.row0 + lane_base < t.row_end) {
#pragma unroll 1
                for (int gi = g_first; gi < g_end; ++gi) {
                    uint32_t v[2][32];
                    tmem_ld32_async(taddr + (uint32_t)(gi * 64), v[0]);
                    tmem_ld32_async(taddr + (uint32_t)(gi * 64 + 32), v[1]);
                    tmem_wait_ld();
                    if constexpr (EPI == EPI_UP) {
                        const int nb = t.n0 / 2 + gi * 32;  // 32 neurons: one block of h
                        float h[32];
                        swiglu16(v[0], h);
                        swiglu16(v[1], h + 16);
                        uint32_t amax = 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (nb + i >= a.n_valid)  // neurons past m (their W rows are not read)
                                h[i] = 0.f;
                            amax = max(amax, __float_as_uint(h[i]) & 0x7fffffffu);
                        }
                        const uint32_t byte = mx4_scale_byte(amax);
                        const float inv = mx4_inverse(byte == 255u ? 0u : byte);
                        uint32_t c[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float q[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                q[i] = h[8 * j + i] * inv;
                            c[j] = byte == 255u ? 0u : mx4_codes8(q);
                        }
                        if (rv && nb < 2 * a.ld) {
                            st_v4(static_cast<uint8_t *>(a.out) + (int64_t)row * a.ld + nb / 2,
                                  make_uint4(c[0], c[1], c[2], c[3]));
                            const int tkh = (2 * a.ld + 127) / 128;
                            uint8_t *sp = a.h_s + mx4_scale_at(mx4_expert_tile(t.off, t.e), tkh,
                                                               row - t.off, nb / 32);
                            sp[0] = (uint8_t)byte;
                            if (nb + 32 >= 2 * a.ld)  // the word's bytes past the last block
                                for (int b = nb / 32 + 1; b % 4 != 0; ++b)
                                    *++sp = 0;
                        }
                    } else if (rv) {
                        bf16 *dst = static_cast<bf16 *>(a.out) + (int64_t)row * a.ld;
#pragma unroll
                        for (int q2 = 0; q2 < 2; ++q2)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int col = t.n0 + gi * 64 + q2 * 32 + q * 8;
                                if (col < a.n_valid) {
                                    float f[8];
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        f[i] = __uint_as_float(v[q2][q * 8 + i]);
                                    st_v4(dst + col, f32x8_to_bf16(f));
                                }
                            }
                    }
                    __syncwarp();  // the next tcgen05.ld takes the whole warp
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&aux->tempty[acc]));
            if (++acc == ACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// ------------------------------------------------------------------------ host side

struct DevInfo {
    int sms = 0;
};
static std::mutex g_mu;
static DevInfo g_dev[64];

static cudaError_t prepare_device(DevInfo **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    DevInfo &di = g_dev[dev];
    if (di.sms == 0) {
        int sms = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(mx4_gemm_kernel<EPI_UP, 192>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Geo<192>::SMEM)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(mx4_gemm_kernel<EPI_DOWN, 192>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Geo<192>::SMEM)) != cudaSuccess)
            return e;
        di.sms = sms;
    }
    *out = &di;
    return cudaSuccess;
}

template <int EPI>
static cudaError_t launch_gemm(const void *A, uint64_t rows, const void *B, const GemmArgs &args,
                               cudaStream_t s)
{
    DevInfo *di = nullptr;
    cudaError_t e = prepare_device(&di);
    if (e != cudaSuccess)
        return e;
    constexpr int BN = 192;
    // code rows as 2-byte elements (four codes each): the maps only copy
    const uint64_t kel = (uint64_t)args.K32 / 4, pitch = (uint64_t)args.K32 / 2;
    CUtensorMap ta, tb;
    const uint64_t da[2] = {kel, rows}, sa[1] = {pitch};
    const uint64_t db[3] = {kel, (uint64_t)args.N, (uint64_t)args.E};
    const uint64_t sb[2] = {pitch, pitch * args.N};
    const uint32_t ba[2] = {BKB / 2, BM}, bb[3] = {BKB / 2, BN, 1};
    if ((e = make_map(&ta, A, 2, da, sa, ba)) != cudaSuccess ||
        (e = make_map(&tb, B, 3, db, sb, bb)) != cudaSuccess)
        return e;
    return launch_pdl(mx4_gemm_kernel<EPI, BN>, dim3(di->sms), dim3(NUM_THREADS), Geo<BN>::SMEM, s,
                      ta, tb, args);
}

}  // namespace mxg

cudaError_t launch_mx4_up(const moe_params_t *p, const void *xq, const void *xs,
                          const int32_t *offsets, const void *W13q, const void *W13s, void *hq,
                          void *hs, int32_t *status, cudaStream_t s)
{
    mxg::GemmArgs a = {};
    a.a_s = (const uint8_t *)xs;
    a.b_s = (const uint8_t *)W13s;
    a.offsets = offsets;
    a.out = hq;
    a.h_s = (uint8_t *)hs;
    a.E = p->E;
    a.N = 2 * round_up(p->m, 16);
    a.K32 = p->d;
    a.n_valid = p->m;
    a.ld = mx4_k32(p->m) / 2;
    a.status = status;
    a.wait_ns = wait_limit_ns();
    count_launch();
    return mxg::launch_gemm<mxg::EPI_UP>(xq, (uint64_t)p->T * p->k, W13q, a, s);
}

cudaError_t launch_mx4_down(const moe_params_t *p, const void *hq, const void *hs,
                            const int32_t *offsets, const void *W2q, const void *W2s, void *out,
                            int32_t *status, cudaStream_t s)
{
    mxg::GemmArgs a = {};
    a.a_s = (const uint8_t *)hs;
    a.b_s = (const uint8_t *)W2s;
    a.offsets = offsets;
    a.out = out;
    a.E = p->E;
    a.N = p->d;
    a.K32 = mx4_k32(p->m);
    a.n_valid = p->d;
    a.ld = p->d;
    a.status = status;
    a.wait_ns = wait_limit_ns();
    count_launch();
    return mxg::launch_gemm<mxg::EPI_DOWN>(hq, (uint64_t)p->T * p->k, W2q, a, s);
}

}  // namespace moe
