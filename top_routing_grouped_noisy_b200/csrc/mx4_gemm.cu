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
// offsets.  A tile's A rows come in boxes of 32, as many as it has: a TMA box costs the copy
// engine 2 to 4 cycles a 128-byte row whether the row exists or not (4 where rows do not start
// on 128-byte lines), and with few rows that bounds the kernel (1 token, 128-row boxes: 0.38 us
// a stage, a third of it W's rows).  TMEM: two accumulators of BN columns, then a set of 24 scale
// columns for each stage.  Roles: warp 0 TMA producer, warp 1 TMEM allocator and issuer, warps
// 2-9 epilogue (each thread one row, half of the columns).
//
// Measured (d 4096, m 1376, 8 experts, top 2; a3 / a4): 1 token 8.1 / 5.3 us (weights 11.9 and
// 6.0 MB), 203 tokens 13.8 / 9.3, 2048 tokens 25.5 / 25.7, 16384 tokens (the pair kernels) 132 /
// 108 in a short run (5.6 and 3.4 PFLOP/s) and 154 / 116 in a long one, under the power cap at
// 1455 / 1690 MHz.
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
constexpr int kABox = 32;           // 1-SM kernel: rows of one A box
constexpr int ACC = 2;
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

template <int EPI, int BN>
struct Geo {
    static constexpr int BT = (BN + 127) / 128;             // B scale tiles of a tile
    static constexpr int A_BYTES = BM * BKB;
    static constexpr int B_BYTES = BN * BKB;
    static constexpr int SFA = 2 * kMx4Tile;                // two K tiles per stage
    static constexpr int SFB = BT * 2 * kMx4Tile;
    static constexpr int STAGE = A_BYTES + B_BYTES + SFA + SFB;
    static constexpr int EPI_BYTES = EPI == EPI_DOWN ? kEpiStageBytes : 0;
    static constexpr int FIXED = 1024 + EPI_BYTES + (int)sizeof(Aux);
    static constexpr int FIT = (227 * 1024 - FIXED) / STAGE;
    static constexpr int STAGES = FIT < kMaxStages ? FIT : kMaxStages;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static constexpr int SF_COL = ACC * BN;
    // a set of scale columns per stage: a full stage's last products, and with them the last
    // use of its set, have completed
    static constexpr int SETS = STAGES;
    // kind::mxf4, A and B e2m1 K-major, e8m0 scales, M = 128
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                      (1u << 23) | ((uint32_t)(BM >> 7) << 27);
    static_assert(BN % 64 == 0 && STAGE % 1024 == 0, "tile");
    static_assert(SF_COL + SETS * kSfCols <= TMEM_COLS, "TMEM columns");
    static_assert(SMEM > 114 * 1024, "one CTA per SM: TMEM is allocated before the grid wait");
};

// The producer and the issuer run their loops as whole warps and let one elected lane issue:
// the loops' values stay in uniform registers, where copies and products take their operands
// (a loop of one lane spent about 450 cycles a stage on moving them, as long as the
// products take).  The warp number is made uniform the same way.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int warp_number()
{
    return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
}

// A wait of a whole warp, with one answer: the lanes' clocks may differ at the limit, and the
// epilogue's tcgen05.ld takes all lanes.  (The producer's and the issuer's waits are followed by
// nothing that does.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                          volatile int32_t *abort_flag, int32_t *status)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns, abort_flag, status));
}

// Descriptors, low and high words (bit 16 of the low word: the leading byte offset, unused by
// the swizzled tiles and absent from the scale tiles').  Operand tiles: K-major, 128-byte swizzle (as tc::sdesc);
// scale tiles: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kSfDescHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t hi)
{
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ void sf_copy(uint32_t tmem, uint64_t sd)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sd) : "memory");
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
    int32_t rows;              // T*k
    int n_valid;               // UP: neurons m; DOWN: columns d
    int ld;                    // DOWN: d; UP: h32 / 2
    int after_up;              // DOWN: the kernel before in the stream is this call's UP
    int32_t *status;
    uint64_t wait_ns;
};

// The offsets and, times `per`, the number of row tiles (ROWS high) before each expert, by one
// warp.  Offsets that no dispatch writes (below 0, above T*k, falling) are reported and taken as
// the nearest that keep every row inside the buffers.
template <int ROWS>
__device__ __forceinline__ void load_offsets(const GemmArgs &a, int32_t *off, int32_t *start, int per)
{
    const int lane = threadIdx.x & 31;
    int32_t top = 0, tiles = 0;  // offset and row tiles up to the 32 experts before
    for (int i0 = 0; i0 <= a.E; i0 += 32) {
        const bool in = i0 + lane <= a.E;
        const int32_t given = in ? a.offsets[i0 + lane] : 0;
        int32_t v = max(top, min(given, a.rows));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
            v = lane >= o ? max(v, u) : v;
        }
        int32_t before = __shfl_up_sync(0xffffffffu, v, 1);
        before = lane == 0 ? (i0 == 0 ? v : top) : before;
        int32_t t = (v - before + ROWS - 1) / ROWS;  // of expert i0 + lane - 1
        t += lane == 0 ? tiles : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, t, o);
            t += lane >= o ? u : 0;
        }
        if (in) {
            if (v != given)
                set_status(a.status, MOE_ERR_DEVICE_BADINDEX);
            off[i0 + lane] = v;
            start[i0 + lane] = t * per;
        }
        top = __shfl_sync(0xffffffffu, v, 31);
        tiles = __shfl_sync(0xffffffffu, t, 31);
    }
    __syncwarp();
}

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

// One block of h (32 neurons from nb on) of this thread's row from its 64 accumulator columns:
// codes and scale byte.  Neurons past m, whose W rows are not read, are zeros.
__device__ __forceinline__ uint4 swiglu_block(const uint32_t (&v)[2][32], int nb, int m, uint32_t &byte)
{
    float h[32];
    swiglu16(v[0], h);
    swiglu16(v[1], h + 16);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (nb + i >= m)
            h[i] = 0.f;
        amax = max(amax, __float_as_uint(h[i]) & 0x7fffffffu);
    }
    byte = mx4_scale_byte(amax);
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
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// The scale byte of a block of h; with the last block, the rest of its word.
__device__ __forceinline__ void store_scale(const GemmArgs &a, const Tile &t, int row, int nb,
                                            uint32_t byte)
{
    const int tkh = (2 * a.ld + 127) / 128;
    uint8_t *sp = a.h_s + mx4_scale_at(mx4_expert_tile(t.off, t.e), tkh, row - t.off, nb / 32);
    sp[0] = (uint8_t)byte;
    if (nb + 32 >= 2 * a.ld)
        for (int b = nb / 32 + 1; b % 4 != 0; ++b)
            *++sp = 0;
}

// 64 output columns from col on of this thread's row: boxes wholly inside the expert's rows
// and the columns through the staging slots, the others per lane.
__device__ __forceinline__ void store_64(const GemmArgs &a, const uint32_t (&v)[2][32], int col0,
                                         int row0, int row, int row_end, EpiStore &st)
{
#pragma unroll
    for (int q2 = 0; q2 < 2; ++q2) {
        const int col = col0 + q2 * 32;
        if (row0 + 32 <= row_end && col + 32 <= a.n_valid) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                pk[i] = pack_bf16x2(__uint_as_float(v[q2][2 * i]), __uint_as_float(v[q2][2 * i + 1]));
            stage_box(st, pk, col, row0);
        } else if (row < row_end) {
            bf16 *dst = static_cast<bf16 *>(a.out) + (int64_t)row * a.ld + col;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (col + q * 8 < a.n_valid) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = __uint_as_float(v[q2][q * 8 + i]);
                    st_v4(dst + q * 8, f32x8_to_bf16(f));
                }
        }
    }
}

template <int EPI, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmO, const __grid_constant__ GemmArgs a)
{
    using G = Geo<EPI, BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Aux *aux = reinterpret_cast<Aux *>(smem + G::STAGES * G::STAGE + G::EPI_BYTES);
    const int warp = warp_number(), lane = threadIdx.x & 31;
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
    // Behind this call's UP, DOWN reads the offsets and its first stages of W before it waits:
    // UP triggers after its own wait, so whatever wrote them has completed by then, and UP
    // itself writes neither.  The first loads then run beside UP's last tiles (the FFN, d 4096,
    // m 1376, 8 experts, top 2: 16.9 to 15.9 us for 1 token, 27.4 to 25.7 us for 203)
    const bool ahead = EPI == EPI_DOWN && a.after_up != 0;
    if (!ahead) {
        pdl_wait();
        pdl_trigger();
    }
    const int n_tiles = (a.N + BN - 1) / BN;
    if (warp == 2) {
        load_offsets<BM>(a, aux->off, aux->tstart, n_tiles);
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
        // -------------------------------------------------------------- TMA producer
        const bool lead = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        int64_t fills = 0;
        bool ok = true;
        int kb0 = 0;  // stages of the first tile that are on their way
        if (ahead) {
            Tile t = {};
            if ((int)blockIdx.x < total) {
                t = decode_tile<BN>(aux, blockIdx.x);
                kb0 = min(num_kb, G::STAGES);
            }
            const int a_boxes = min(BM / kABox, (t.row_end - t.row0 + kABox - 1) / kABox);
            const int nbt = min(G::BT, trb - t.n0 / 128);
            const uint8_t *sa_src =
                a.a_s + (mx4_expert_tile(t.off, t.e) + (t.row0 - t.off) / BM) * tk * kMx4Tile;
            const uint8_t *sb_src = a.b_s + ((int64_t)t.e * trb + t.n0 / 128) * tk * kMx4Tile;
            for (int half = 0; half < 2; ++half) {  // W's side, the wait, the rows' side
                for (int kb = 0; kb < kb0; ++kb) {
                    const uint32_t fb = smem_u32(&aux->full[kb]);
                    const uint32_t sa = smem_base + kb * G::STAGE, sb = sa + G::A_BYTES;
                    const uint32_t sfa = sb + G::B_BYTES, sfb = sfa + G::SFA;
                    const uint32_t kt = (uint32_t)min(2, tk - 2 * kb) * kMx4Tile;
                    if (lead && half == 0) {
                        mbar_expect_tx(fb, (uint32_t)(a_boxes * kABox * BKB + G::B_BYTES) + kt * (1 + nbt));
                        tma_load_3d(&tmB, fb, sb, kb * (BKB / 2), t.n0, t.e);
                        for (int i = 0; i < nbt; ++i)
                            bulk_load(sfb + i * 2 * kMx4Tile,
                                      sb_src + ((int64_t)i * tk + 2 * kb) * kMx4Tile, kt, fb);
                    } else if (lead) {
                        for (int i = 0; i < a_boxes; ++i)
                            tma_load_2d(&tmA, fb, sa + i * kABox * BKB, kb * (BKB / 2), t.row0 + i * kABox);
                        bulk_load(sfa, sa_src + (int64_t)2 * kb * kMx4Tile, kt, fb);
                    }
                }
                if (half == 0) {
                    pdl_wait();
                    pdl_trigger();
                }
            }
            fills = kb0;
            stage = kb0 % G::STAGES;
            phase = kb0 == G::STAGES;
        }
        for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
            const Tile t = decode_tile<BN>(aux, tile);
            // rows past the expert's are not loaded: the products read what the stage held, and
            // only make accumulator rows nobody stores
            const int a_boxes = min(BM / kABox, (t.row_end - t.row0 + kABox - 1) / kABox);
            const uint8_t *sa_src =
                a.a_s + (mx4_expert_tile(t.off, t.e) + (t.row0 - t.off) / BM) * tk * kMx4Tile;
            const int nb0 = t.n0 / 128;
            const int nbt = min(G::BT, trb - nb0);  // B scale tiles that exist
            const uint8_t *sb_src = a.b_s + ((int64_t)t.e * trb + nb0) * tk * kMx4Tile;
            for (int kb = kb0; kb < num_kb; ++kb) {
                if (!mbar_wait(smem_u32(&aux->empty[stage]), phase ^ 1u, a.wait_ns, abort_flag,
                               a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = smem_u32(&aux->full[stage]);
                const uint32_t sa = smem_base + stage * G::STAGE, sb = sa + G::A_BYTES;
                const uint32_t sfa = sb + G::B_BYTES, sfb = sfa + G::SFA;
                const uint32_t kt = (uint32_t)min(2, tk - 2 * kb) * kMx4Tile;
                if (lead) {
                    mbar_expect_tx(fb, (uint32_t)(a_boxes * kABox * BKB + G::B_BYTES) + kt * (1 + nbt));
                    for (int i = 0; i < a_boxes; ++i)
                        tma_load_2d(&tmA, fb, sa + i * kABox * BKB, kb * (BKB / 2), t.row0 + i * kABox);
                    tma_load_3d(&tmB, fb, sb, kb * (BKB / 2), t.n0, t.e);
                    bulk_load(sfa, sa_src + (int64_t)2 * kb * kMx4Tile, kt, fb);
                    for (int i = 0; i < nbt; ++i)
                        bulk_load(sfb + i * 2 * kMx4Tile,
                                  sb_src + ((int64_t)i * tk + 2 * kb) * kMx4Tile, kt, fb);
                }
                ++fills;
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            kb0 = 0;
        }
        for (int s = 0; s < G::STAGES; ++s) {
            const int64_t n = fills / G::STAGES + (s < fills % G::STAGES ? 1 : 0);
            if (n > 0)
                mbar_drain(smem_u32(&aux->full[s]), (uint32_t)((n - 1) & 1));
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- issuer
        if (ahead)
            pdl_wait();  // its waits have a time limit: none of it goes to the kernel before
        const bool lead = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        const int nk = (a.K32 + 63) / 64;  // products along K
        const uint32_t lo0 = desc_lo(smem_base);
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
                if (!mbar_wait(smem_u32(&aux->full[stage]), phase, a.wait_ns, abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t la = lo0 + (uint32_t)(stage * (G::STAGE >> 4));
                const uint32_t lb = la + (G::A_BYTES >> 4);
                const uint32_t lsa = lb + (G::B_BYTES >> 4) - (1u << 16), lsb = lsa + (G::SFA >> 4);
                const uint32_t sf = tmem_base + (uint32_t)(G::SF_COL + stage * kSfCols);
                const int halves = min(2, tk - 2 * kb), ks = min(4, nk - 4 * kb);
                if (lead) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        if (hh < halves) {
                            sf_copy(sf + hh * 12, desc(lsa + hh * (kMx4Tile >> 4), kSfDescHi));
#pragma unroll
                            for (int i = 0; i < G::BT; ++i)
                                sf_copy(sf + hh * 12 + 4 + i * 4,
                                        desc(lsb + (i * 2 + hh) * (kMx4Tile >> 4), kSfDescHi));
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < ks) {
                            const uint32_t id = (uint32_t)(k & 1) * 2u, col = sf + (uint32_t)(k >> 1) * 12;
                            umma_mx4(d_tmem, desc(la + 2 * k, kDescHi), desc(lb + 2 * k, kDescHi),
                                     G::IDESC | (id << 4) | (id << 29), col, col + 4 + b_shift,
                                     (kb | k) != 0);
                        }
                    umma_commit(smem_u32(&aux->empty[stage]));
                }
                if (++stage == G::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            if (lead)
                umma_commit(smem_u32(&aux->tfull[acc]));
            if (++acc == ACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (lead)
            umma_commit(smem_u32(&aux->drain));
        mbar_drain(smem_u32(&aux->drain), 0);
    } else {
        // -------------------------------------------------------------- epilogue
        if (ahead)
            pdl_wait();
        const int lane_base = (warp & 3) * 32;
        const bool upper = (warp - 2) / 4 != 0;
        // 64-column groups of the tile: the first half of the warps takes the larger half
        constexpr int kGroups = BN / 64, kHalf0 = (kGroups + 1) / 2;
        const int g_first = upper ? kHalf0 : 0, g_end = upper ? kGroups : kHalf0;
        EpiStore st{&tmO, smem_base + (uint32_t)(G::STAGES * G::STAGE + (warp - 2) * 2 * kStageSlotBytes), 0};
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
            const Tile t = decode_tile<BN>(aux, tile);
            if (!warp_wait(smem_u32(&aux->tfull[acc]), acc_phase, a.wait_ns, abort_flag, a.status))
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
                        uint32_t byte;
                        const uint4 c = swiglu_block(v, nb, a.n_valid, byte);
                        if (rv && nb < 2 * a.ld) {
                            st_v4(static_cast<uint8_t *>(a.out) + (int64_t)row * a.ld + nb / 2, c);
                            store_scale(a, t, row, nb, byte);
                        }
                    } else {
                        store_64(a, v, t.n0 + gi * 64, t.row0 + lane_base, row, t.row_end, st);
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
        if (lane == 0)
            bulk_wait_all();  // this lane's output stores are done before the CTA exits
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// ------------------------------------------------------------------------ 2-SM variant
// cta_group::2: a cluster of two CTAs owns a 256 x 256 tile.  CTA r loads rows [128r, 128r +
// 128) of A and of B with A's scales for its rows and B's for all 256 (every CTA's
// accumulators see all columns); the leader issues M = 256 products.  The 1-SM kernel copies 320
// rows for 128 x 192 x 256 of work; here 256 rows serve 128 x 256 x 256 of each SM's.
// UP of 16384 tokens: 5.6 PFLOP/s in a short run, 84% of four times the measured bf16 rate; in a
// long one 154 us x 1455 MHz (sampled) = 224 thousand cycles for the 1250 products of 256 x 256 x 64
// that a pair issues, 180 each, where 16384 multiply-adds a cycle and SM would take 128.
//
// TMEM.  Two 256-column accumulators do not leave room for scales, so they share 64 columns:
// accumulator 0 is columns 0..255, accumulator 1 columns 192..447, scales 448..471 and 480..503
// (two sets).
// The epilogue reads the shared 64 columns first and then lets the next tile's products
// start; the tile before (the same accumulator) is read by then, since every warp takes the
// tiles in order.  A set of scales is copied over only after the products of two stages ago
// have completed (its empty barrier), so nothing rests on the order of copies after products.
//   full[s]   leader: both CTAs' bytes          empty[s]  both CTAs: the leader's commit
//   tfull[a]  both CTAs: the leader's commit    tfree     leader: 8 epilogue warps of each CTA
// Loads carry no multicast qualifier.
namespace pair {

constexpr int BN = 256;
constexpr int BNH = 128;
constexpr int A_BYTES = BM * BKB;
constexpr int B_BYTES = BNH * BKB;
constexpr int SFA = 2 * kMx4Tile;
constexpr int SFB = 2 * 2 * kMx4Tile;
constexpr int STAGE = A_BYTES + B_BYTES + SFA + SFB;
constexpr int ACC_STEP = 192;              // accumulator 1 starts here
constexpr int SF_COL = ACC_STEP + BN;      // 448
constexpr uint64_t kAbortSettleNs = 200000ull;
constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) |
                            ((uint32_t)(256 >> 7) << 27);
static_assert(SF_COL + 32 + kSfCols <= TMEM_COLS, "TMEM columns");
static_assert(STAGE % 1024 == 0, "stage alignment");

template <int EPI>
struct Geo {
    static constexpr int EPI_BYTES = EPI == EPI_DOWN ? kEpiStageBytes : 0;
    static constexpr int STAGES = EPI == EPI_DOWN ? 5 : 6;
};

struct Aux {
    uint64_t full[6];
    uint64_t empty[6];
    uint64_t tfull[2];
    uint64_t tfree;
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t off[MOE_MAX_EXPERTS + 1];
    int32_t tstart[MOE_MAX_EXPERTS + 1];
};
template <int EPI>
constexpr int smem_bytes() { return 1024 + Geo<EPI>::STAGES * STAGE + Geo<EPI>::EPI_BYTES + (int)sizeof(Aux); }
static_assert(smem_bytes<EPI_UP>() <= 227 * 1024 && smem_bytes<EPI_DOWN>() <= 227 * 1024, "shared memory");

__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Relaxed: what the arrival hands over is accumulator columns, ordered by hand_over's fence.  A
// release would first wait for this thread's stores of h or of the last output tile, about
// 700 ns in which no products run.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}
// The warp hands back the accumulator columns it has loaded so far: every lane's tcgen05.ld (over
// by tcgen05.wait::ld) is ordered before the arrival by the fence.
__device__ __forceinline__ void hand_over(uint32_t cluster_addr)
{
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive_cluster(cluster_addr);
}
__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t cluster_addr)
{
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}
__device__ __forceinline__ void load_2d(const CUtensorMap *map, uint32_t bar_cluster, uint32_t dst,
                                        int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void load_3d(const CUtensorMap *map, uint32_t bar_cluster, uint32_t dst,
                                        int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// scale tile to the TMEM of both CTAs, each from its own shared memory
__device__ __forceinline__ void sf_copy(uint32_t tmem, uint64_t sd)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sd) : "memory");
}
__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t sfa, uint32_t sfb, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit_both(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void commit_own(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}

// Tile order inside an expert: bands of `band` row tiles, row tiles fastest inside a band,
// then the band's column tiles (as in the bf16 pair kernel).
__device__ __forceinline__ Tile decode(const Aux *aux, int tile, int n_tiles, int band)
{
    Tile t;
    int e = 0;
    while (tile >= aux->tstart[e + 1])
        ++e;
    const int local = tile - aux->tstart[e];
    const int rows = aux->off[e + 1] - aux->off[e];
    const int mtiles = (rows + 2 * BM - 1) / (2 * BM);
    int G = (band > 0 && band < mtiles) ? band : mtiles;
    const int nbands = (mtiles + G - 1) / G;
    G = (mtiles + nbands - 1) / nbands;
    const int bi = local / (G * n_tiles);
    const int rem = local - bi * G * n_tiles;
    const int gr = mtiles - bi * G < G ? mtiles - bi * G : G;
    t.e = e;
    t.off = aux->off[e];
    t.row0 = t.off + (bi * G + rem % gr) * 2 * BM;
    t.row_end = aux->off[e + 1];
    t.n0 = rem / gr * BN;
    return t;
}

template <int EPI>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    mx4_gemm_2sm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSA,
                        const __grid_constant__ CUtensorMap tmSB,
                        const __grid_constant__ CUtensorMap tmO, const __grid_constant__ GemmArgs a,
                        int band)
{
    constexpr int STAGES = Geo<EPI>::STAGES;
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Aux *aux = reinterpret_cast<Aux *>(smem + STAGES * STAGE + Geo<EPI>::EPI_BYTES);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    volatile int32_t *abort_flag = &aux->abort_flag;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    const int cluster_id = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&aux->full[s]), 1);
            mbar_init(smem_u32(&aux->empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i)
            mbar_init(smem_u32(&aux->tfull[i]), 1);
        mbar_init(smem_u32(&aux->tfree), 2 * EPI_WARPS);
        mbar_init(smem_u32(&aux->drain), 1);
        aux->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        const CUtensorMap *maps[5] = {&tmA, &tmB, &tmSA, &tmSB, &tmO};
        for (int i = 0; i < (EPI == EPI_DOWN ? 5 : 4); ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
    }
    const int n_tiles = (a.N + BN - 1) / BN;
    if (warp == 2) {
        load_offsets<2 * BM>(a, aux->off, aux->tstart, n_tiles);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&aux->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    const uint32_t tmem_base = aux->tmem_base;
    const int total = aux->tstart[a.E];
    const int num_kb = (a.K32 + BKC - 1) / BKC;
    const int trb = (a.N + 127) / 128;
    const uint32_t smem_base = smem_u32(smem);

    if (warp == 0) {
        // -------------------------------------------------------------- TMA producer (both)
        const bool lead = elect_one();
        const uint32_t full0 = map_rank(smem_u32(&aux->full[0]), 0);
        int stage = 0;
        uint32_t phase = 0;
        int64_t fills = 0;
        bool ok = true;
        for (int tile = cluster_id; tile < total && ok; tile += nclusters) {
            const Tile t = decode(aux, tile, n_tiles, band);
            const int a_row = t.row0 + (int)rank * BM, b_row = t.n0 + (int)rank * BNH;
            const int sa_row = (int)mx4_expert_tile(t.off, t.e) + (t.row0 - t.off) / BM + (int)rank;
            const int sb_row = t.e * trb + t.n0 / 128;
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!mbar_wait(smem_u32(&aux->empty[stage]), phase ^ 1u, a.wait_ns, abort_flag,
                               a.status)) {
                    ok = false;
                    break;
                }
                const uint32_t fb0 = full0 + 8 * stage;
                const uint32_t sa = smem_base + stage * STAGE, sb = sa + A_BYTES;
                if (lead) {
                    if (leader)
                        mbar_expect_tx(smem_u32(&aux->full[stage]), 2 * STAGE);
                    load_2d(&tmA, fb0, sa, kb * (BKB / 2), a_row);
                    load_3d(&tmB, fb0, sb, kb * (BKB / 2), b_row, t.e);
                    load_2d(&tmSA, fb0, sb + B_BYTES, kb * 256, sa_row);
                    load_2d(&tmSB, fb0, sb + B_BYTES + SFA, kb * 256, sb_row);
                }
                ++fills;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (leader)  // the leader's full barriers count both CTAs' bytes
            for (int s = 0; s < STAGES; ++s) {
                const int64_t n = fills / STAGES + (s < fills % STAGES ? 1 : 0);
                if (n > 0)
                    mbar_drain(smem_u32(&aux->full[s]), (uint32_t)((n - 1) & 1));
            }
    } else if (warp == 1) {
        if (leader) {
            // ---------------------------------------------------------- issuer (leader)
            const bool lead = elect_one();
            int stage = 0;
            uint32_t phase = 0;
            int old = STAGES - 2;    // the stage issued two before this one, and its phase
            uint32_t old_phase = 1;
            uint32_t set = 0;
            int ti = 0;              // tiles issued
            bool ok = true, first = true;
            const int nk = (a.K32 + 63) / 64;
            const uint32_t lo0 = desc_lo(smem_base);
            for (int tile = cluster_id; tile < total && ok; tile += nclusters, ++ti) {
                // the shared columns of the tile before have been read
                if (ti > 0 && !mbar_wait(smem_u32(&aux->tfree), (uint32_t)(ti - 1) & 1u, a.wait_ns,
                                         abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)((ti & 1) * ACC_STEP);
                for (int kb = 0; kb < num_kb; ++kb) {
                    // the products of two stages ago are done with this set of scales (before
                    // the third stage there are none)
                    if (!mbar_wait(smem_u32(&aux->full[stage]), phase, a.wait_ns, abort_flag,
                                   a.status) ||
                        (!first && !mbar_wait(smem_u32(&aux->empty[old]), old_phase, a.wait_ns,
                                              abort_flag, a.status))) {
                        ok = false;
                        break;
                    }
                    const uint32_t la = lo0 + (uint32_t)(stage * (STAGE >> 4));
                    const uint32_t lb = la + (A_BYTES >> 4);
                    const uint32_t lsa = lb + (B_BYTES >> 4) - (1u << 16), lsb = lsa + (SFA >> 4);
                    const uint32_t sf = tmem_base + SF_COL + set;
                    const int ks = min(4, nk - 4 * kb);
                    if (lead) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            sf_copy(sf + hh * 12, desc(lsa + hh * (kMx4Tile >> 4), kSfDescHi));
                            sf_copy(sf + hh * 12 + 4, desc(lsb + hh * (kMx4Tile >> 4), kSfDescHi));
                            sf_copy(sf + hh * 12 + 8, desc(lsb + (2 + hh) * (kMx4Tile >> 4), kSfDescHi));
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < ks) {
                                const uint32_t id = (uint32_t)(k & 1) * 2u;
                                const uint32_t col = sf + (uint32_t)(k >> 1) * 12;
                                umma(d_tmem, desc(la + 2 * k, kDescHi), desc(lb + 2 * k, kDescHi),
                                     kIdesc | (id << 4) | (id << 29), col, col + 4, (kb | k) != 0);
                            }
                        commit_both(smem_u32(&aux->empty[stage]));
                    }
                    set ^= 32u;
                    if (++old == STAGES) {
                        old = 0;
                        old_phase ^= 1u;
                        first = false;
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                if (lead)
                    commit_both(smem_u32(&aux->tfull[ti & 1]));
            }
            if (lead)
                commit_own(smem_u32(&aux->drain));
            mbar_drain(smem_u32(&aux->drain), 0);
        }
    } else {
        // -------------------------------------------------------------- epilogue (both)
        const int lane_base = (warp & 3) * 32;
        const int half = (warp - 2) / 4;  // 64-column groups 2 half, 2 half + 1
        const uint32_t tfree0 = map_rank(smem_u32(&aux->tfree), 0);
        EpiStore st{&tmO, smem_base + (uint32_t)(STAGES * STAGE + (warp - 2) * 2 * kStageSlotBytes), 0};
        int ti = 0;
        for (int tile = cluster_id; tile < total; tile += nclusters, ++ti) {
            const Tile t = decode(aux, tile, n_tiles, band);
            const int acc = ti & 1;
            if (!warp_wait(smem_u32(&aux->tfull[acc]), (uint32_t)(ti >> 1) & 1u, a.wait_ns, abort_flag,
                           a.status))
                break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)lane_base << 16) + (uint32_t)(acc * ACC_STEP);
            const int row0 = t.row0 + (int)rank * BM + lane_base, row = row0 + lane;
            const bool rv = row < t.row_end;
            // the shared columns are group 3 of accumulator 0 and group 0 of accumulator 1: the
            // half that has them takes them first
            const bool shares = half == 1 - acc;
            if (!shares)  // for the issuer: this warp has read the tile before
                hand_over(tfree0);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int gi = 2 * half + ((acc == 0 && half == 1) ? 1 - i : i);
                uint32_t v[2][32];
                tmem_ld32_async(taddr + (uint32_t)(gi * 64), v[0]);
                tmem_ld32_async(taddr + (uint32_t)(gi * 64 + 32), v[1]);
                tmem_wait_ld();
                if (shares && i == 0)
                    hand_over(tfree0);
                if constexpr (EPI == EPI_UP) {
                    const int nb = t.n0 / 2 + gi * 32;  // 32 neurons: one block of h
                    uint32_t byte;
                    const uint4 c = swiglu_block(v, nb, a.n_valid, byte);
                    if (rv && nb < 2 * a.ld) {
                        st_v4(static_cast<uint8_t *>(a.out) + (int64_t)row * a.ld + nb / 2, c);
                        store_scale(a, t, row, nb, byte);
                    }
                } else {
                    store_64(a, v, t.n0 + gi * 64, row0, row, t.row_end, st);
                }
                __syncwarp();  // the next tcgen05.ld takes the whole warp
            }
        }
        if (lane == 0)
            bulk_wait_all();  // this lane's output stores are done before the CTA exits
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    // after an abort, give copies still in flight time to land before either CTA of
    // the pair releases its shared memory (the other CTA's loads signal the leader)
    if (threadIdx.x == 0) {
        const int peer_abort = ld_cluster_s32(map_rank(smem_u32(&aux->abort_flag), rank ^ 1u));
        if (*abort_flag || peer_abort) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kAbortSettleNs) {
            }
        }
    }
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

// ------------------------------------------------------------------------ resident A
// The second product has few stages along K (at most kResKb) and, per stage, 256 rows to load
// for 256 x 256 x 256 of work; with m = 1376 they do not start on 128-byte lines and take about
// twice the copy engine's time of those that do.  Here a pair keeps the A rows of its tile, all
// of K, in shared memory while it walks over a chunk of column tiles, so only B is loaded per
// stage.  A's K blocks are freed one by one by the chunk's last tile (aempty) and refilled for the next one behind it.  Measured, with
// the kernel above / this one: 16384 tokens (d 4096, m 1376, top 2) 119.5 / 106 us, 4096 tokens
// (16 experts, m 688, top 4) 40.4 / 38 us.
//   afull[kb]  leader: both CTAs' bytes      aempty[kb]  both CTAs: the leader's commit
constexpr int kResKb = 6;
constexpr int RES_STAGE = B_BYTES + SFB;   // 18 KB
constexpr int RES_A = A_BYTES + SFA;       // one K block of A, 17 KB
constexpr int kMaxResStages = 7;

struct ResAux {
    uint64_t full[kMaxResStages];
    uint64_t empty[kMaxResStages];
    uint64_t afull[kResKb];
    uint64_t aempty[kResKb];
    uint64_t tfull[2];
    uint64_t tfree;
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t off[MOE_MAX_EXPERTS + 1];
    int32_t ustart[MOE_MAX_EXPERTS + 1];
    int32_t chunk;
};
inline int res_stages(int num_kb)
{
    const int left = 227 * 1024 - 1024 - kEpiStageBytes - (int)sizeof(ResAux) - num_kb * RES_A;
    const int n = left / RES_STAGE;
    return n < kMaxResStages ? n : kMaxResStages;
}
inline int res_smem(int num_kb)
{
    return 1024 + kEpiStageBytes + (int)sizeof(ResAux) + num_kb * RES_A + res_stages(num_kb) * RES_STAGE;
}

// A unit: row tile and chunk of column tiles [n_lo, n_hi) of expert e.
struct ResUnit {
    int e, row0, row_end, off, n_lo, n_hi;
};
__device__ __forceinline__ ResUnit res_unit(const ResAux *aux, int unit, int n_tiles, int nchunks)
{
    ResUnit u;
    int e = 0;
    while (unit >= aux->ustart[e + 1])
        ++e;
    const int local = unit - aux->ustart[e];
    const int mt = local / nchunks, c = local - mt * nchunks;
    u.e = e;
    u.off = aux->off[e];
    u.row0 = u.off + mt * 2 * BM;
    u.row_end = aux->off[e + 1];
    u.n_lo = c * aux->chunk;
    u.n_hi = min(n_tiles, u.n_lo + aux->chunk);
    return u;
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    mx4_down_res_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSA,
                        const __grid_constant__ CUtensorMap tmSB,
                        const __grid_constant__ CUtensorMap tmO, const __grid_constant__ GemmArgs a,
                        int stages)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int num_kb = (a.K32 + BKC - 1) / BKC;
    const int ring = num_kb * RES_A, epi = ring + stages * RES_STAGE;
    ResAux *aux = reinterpret_cast<ResAux *>(smem + epi + kEpiStageBytes);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    volatile int32_t *abort_flag = &aux->abort_flag;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    const int cluster_id = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&aux->full[s]), 1);
            mbar_init(smem_u32(&aux->empty[s]), 1);
        }
        for (int kb = 0; kb < num_kb; ++kb) {
            mbar_init(smem_u32(&aux->afull[kb]), 1);
            mbar_init(smem_u32(&aux->aempty[kb]), 1);
        }
        for (int i = 0; i < 2; ++i)
            mbar_init(smem_u32(&aux->tfull[i]), 1);
        mbar_init(smem_u32(&aux->tfree), 2 * EPI_WARPS);
        mbar_init(smem_u32(&aux->drain), 1);
        aux->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        const CUtensorMap *maps[5] = {&tmA, &tmB, &tmSA, &tmSB, &tmO};
        for (int i = 0; i < 5; ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[i])) : "memory");
    }
    const int n_tiles = (a.N + BN - 1) / BN;
    if (warp == 2) {
        load_offsets<2 * BM>(a, aux->off, aux->ustart, 1);
        // column tiles per chunk, 1 << lane: the fewest loads on the busiest pair, A counting as
        // much as one column tile's B; the smaller of equal ones
        const int mt = aux->ustart[a.E], c = 1 << min(lane, 4);
        const int64_t units = (int64_t)mt * ((n_tiles + c - 1) / c);
        int64_t best = ((units + nclusters - 1) / nclusters * (min(c, n_tiles) + 1) << 5) + c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        const int chunk = (int)(best & 31), nchunks = (n_tiles + chunk - 1) / chunk;
        for (int i = lane; i <= a.E; i += 32)
            aux->ustart[i] *= nchunks;
        if (lane == 0)
            aux->chunk = chunk;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&aux->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    const uint32_t tmem_base = aux->tmem_base;
    const int total = aux->ustart[a.E];
    const int nchunks = (n_tiles + aux->chunk - 1) / aux->chunk;
    const int trb = (a.N + 127) / 128;
    const uint32_t smem_base = smem_u32(smem);

    if (warp == 0) {
        // -------------------------------------------------------------- TMA producer (both)
        const bool lead = elect_one();
        const uint32_t full0 = map_rank(smem_u32(&aux->full[0]), 0);
        const uint32_t afull0 = map_rank(smem_u32(&aux->afull[0]), 0);
        int stage = 0, nu = 0;
        uint32_t phase = 0;
        int64_t fills = 0;
        bool ok = true;
        int a_fills = 0;  // K blocks of A issued
        for (int unit = cluster_id; unit < total && ok; unit += nclusters, ++nu) {
            const ResUnit u = res_unit(aux, unit, n_tiles, nchunks);
            const int a_row = u.row0 + (int)rank * BM;
            const int sa_row = (int)mx4_expert_tile(u.off, u.e) + (u.row0 - u.off) / BM + (int)rank;
            for (int nt = u.n_lo; nt < u.n_hi && ok; ++nt) {
                const int b_row = nt * BN + (int)rank * BNH, sb_row = u.e * trb + nt * (BN / 128);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (nt == u.n_lo) {
                        if (!mbar_wait(smem_u32(&aux->aempty[kb]), (uint32_t)(nu & 1) ^ 1u, a.wait_ns,
                                       abort_flag, a.status)) {
                            ok = false;
                            break;
                        }
                        if (lead) {
                            const uint32_t sa = smem_base + kb * RES_A, fb0 = afull0 + 8 * kb;
                            if (leader)
                                mbar_expect_tx(smem_u32(&aux->afull[kb]), 2 * RES_A);
                            load_2d(&tmA, fb0, sa, kb * (BKB / 2), a_row);
                            load_2d(&tmSA, fb0, sa + A_BYTES, kb * 256, sa_row);
                        }
                        ++a_fills;
                    }
                    if (!mbar_wait(smem_u32(&aux->empty[stage]), phase ^ 1u, a.wait_ns, abort_flag,
                                   a.status)) {
                        ok = false;
                        break;
                    }
                    if (lead) {
                        const uint32_t sb = smem_base + ring + stage * RES_STAGE, fb0 = full0 + 8 * stage;
                        if (leader)
                            mbar_expect_tx(smem_u32(&aux->full[stage]), 2 * RES_STAGE);
                        load_3d(&tmB, fb0, sb, kb * (BKB / 2), b_row, u.e);
                        load_2d(&tmSB, fb0, sb + B_BYTES, kb * 256, sb_row);
                    }
                    ++fills;
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        if (leader) {  // the leader's full barriers count both CTAs' bytes
            for (int s = 0; s < stages; ++s) {
                const int64_t n = fills / stages + (s < fills % stages ? 1 : 0);
                if (n > 0)
                    mbar_drain(smem_u32(&aux->full[s]), (uint32_t)((n - 1) & 1));
            }
            for (int kb = 0; kb < num_kb; ++kb) {
                const int n = a_fills / num_kb + (kb < a_fills % num_kb ? 1 : 0);
                if (n > 0)
                    mbar_drain(smem_u32(&aux->afull[kb]), (uint32_t)((n - 1) & 1));
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------------------------------------------------- issuer (leader)
            const bool lead = elect_one();
            int stage = 0, nu = 0;
            uint32_t phase = 0;
            int old = stages - 2;    // the stage issued two before this one, and its phase
            uint32_t old_phase = 1;
            uint32_t set = 0;
            int ti = 0;              // tiles issued
            bool ok = true, first = true;
            const int nk = (a.K32 + 63) / 64;
            const uint32_t lo0 = desc_lo(smem_base);
            for (int unit = cluster_id; unit < total && ok; unit += nclusters, ++nu) {
                const ResUnit u = res_unit(aux, unit, n_tiles, nchunks);
                for (int nt = u.n_lo; nt < u.n_hi && ok; ++nt, ++ti) {
                    // the shared columns of the tile before have been read
                    if (ti > 0 && !mbar_wait(smem_u32(&aux->tfree), (uint32_t)(ti - 1) & 1u, a.wait_ns,
                                             abort_flag, a.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)((ti & 1) * ACC_STEP);
                    for (int kb = 0; kb < num_kb; ++kb) {
                        // with the products of two stages ago done this set of scales is free
                        if ((nt == u.n_lo && !mbar_wait(smem_u32(&aux->afull[kb]), (uint32_t)nu & 1u,
                                                        a.wait_ns, abort_flag, a.status)) ||
                            !mbar_wait(smem_u32(&aux->full[stage]), phase, a.wait_ns, abort_flag,
                                       a.status) ||
                            (!first && !mbar_wait(smem_u32(&aux->empty[old]), old_phase, a.wait_ns,
                                                  abort_flag, a.status))) {
                            ok = false;
                            break;
                        }
                        const uint32_t la = lo0 + (uint32_t)(kb * (RES_A >> 4));
                        const uint32_t lb = lo0 + (uint32_t)((ring + stage * RES_STAGE) >> 4);
                        const uint32_t lsa = la + (A_BYTES >> 4) - (1u << 16);
                        const uint32_t lsb = lb + (B_BYTES >> 4) - (1u << 16);
                        const uint32_t sf = tmem_base + SF_COL + set;
                        const int ks = min(4, nk - 4 * kb);
                        if (lead) {
#pragma unroll
                            for (int hh = 0; hh < 2; ++hh) {
                                sf_copy(sf + hh * 12, desc(lsa + hh * (kMx4Tile >> 4), kSfDescHi));
                                sf_copy(sf + hh * 12 + 4, desc(lsb + hh * (kMx4Tile >> 4), kSfDescHi));
                                sf_copy(sf + hh * 12 + 8, desc(lsb + (2 + hh) * (kMx4Tile >> 4), kSfDescHi));
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < ks) {
                                    const uint32_t id = (uint32_t)(k & 1) * 2u;
                                    const uint32_t col = sf + (uint32_t)(k >> 1) * 12;
                                    umma(d_tmem, desc(la + 2 * k, kDescHi), desc(lb + 2 * k, kDescHi),
                                         kIdesc | (id << 4) | (id << 29), col, col + 4, (kb | k) != 0);
                                }
                            commit_both(smem_u32(&aux->empty[stage]));
                            if (nt + 1 == u.n_hi)
                                commit_both(smem_u32(&aux->aempty[kb]));
                        }
                        set ^= 32u;
                        if (++old == stages) {
                            old = 0;
                            old_phase ^= 1u;
                            first = false;
                        }
                        if (++stage == stages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok)
                        break;
                    if (lead)
                        commit_both(smem_u32(&aux->tfull[ti & 1]));
                }
            }
            if (lead)
                commit_own(smem_u32(&aux->drain));
            mbar_drain(smem_u32(&aux->drain), 0);
        }
    } else {
        // -------------------------------------------------------------- epilogue (both)
        const int lane_base = (warp & 3) * 32;
        const int half = (warp - 2) / 4;  // 64-column groups 2 half, 2 half + 1
        const uint32_t tfree0 = map_rank(smem_u32(&aux->tfree), 0);
        EpiStore st{&tmO, smem_base + (uint32_t)(epi + (warp - 2) * 2 * kStageSlotBytes), 0};
        int ti = 0;
        bool ok = true;
        for (int unit = cluster_id; unit < total && ok; unit += nclusters) {
            const ResUnit u = res_unit(aux, unit, n_tiles, nchunks);
            const int row0 = u.row0 + (int)rank * BM + lane_base, row = row0 + lane;
            for (int nt = u.n_lo; nt < u.n_hi; ++nt, ++ti) {
                const int acc = ti & 1;
                if (!warp_wait(smem_u32(&aux->tfull[acc]), (uint32_t)(ti >> 1) & 1u, a.wait_ns, abort_flag,
                               a.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr =
                    tmem_base + ((uint32_t)lane_base << 16) + (uint32_t)(acc * ACC_STEP);
                const bool shares = half == 1 - acc;  // as in the kernel above
                if (!shares)
                    hand_over(tfree0);
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    const int gi = 2 * half + ((acc == 0 && half == 1) ? 1 - i : i);
                    uint32_t v[2][32];
                    tmem_ld32_async(taddr + (uint32_t)(gi * 64), v[0]);
                    tmem_ld32_async(taddr + (uint32_t)(gi * 64 + 32), v[1]);
                    tmem_wait_ld();
                    if (shares && i == 0)
                        hand_over(tfree0);
                    store_64(a, v, nt * BN + gi * 64, row0, row, u.row_end, st);
                    __syncwarp();  // the next tcgen05.ld takes the whole warp
                }
            }
        }
        if (lane == 0)
            bulk_wait_all();  // this lane's output stores are done before the CTA exits
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    if (threadIdx.x == 0) {  // after an abort, as in the kernel above
        const int peer_abort = ld_cluster_s32(map_rank(smem_u32(&aux->abort_flag), rank ^ 1u));
        if (*abort_flag || peer_abort) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kAbortSettleNs) {
            }
        }
    }
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(TMEM_COLS)
                     : "memory");
    }
}

}  // namespace pair

// ------------------------------------------------------------------------ host side

struct DevInfo {
    int sms = 0;
    int pair_clusters = 0;
};
static std::mutex g_mu;
static DevInfo g_dev[64];

template <typename Kern>
static cudaError_t allow_smem(Kern kern, int bytes)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int BN>
static cudaError_t allow_smem_1sm()
{
    const cudaError_t e = allow_smem(mx4_gemm_kernel<EPI_UP, BN>, Geo<EPI_UP, BN>::SMEM);
    return e != cudaSuccess ? e : allow_smem(mx4_gemm_kernel<EPI_DOWN, BN>, Geo<EPI_DOWN, BN>::SMEM);
}

static void cluster_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int clusters, int smem,
                           cudaStream_t s)
{
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->gridDim = dim3(2 * clusters);
    cfg->blockDim = dim3(NUM_THREADS);
    cfg->dynamicSmemBytes = smem;
    cfg->stream = s;
    cfg->attrs = attr;
    cfg->numAttrs = 2;
}

// SM count, shared-memory opt-in of the kernels, clusters of the pair kernel that fit at once
// (per device, cached)
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
        int sms = 0, n = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = allow_smem_1sm<128>()) != cudaSuccess || (e = allow_smem_1sm<192>()) != cudaSuccess ||
            (e = allow_smem(pair::mx4_gemm_2sm_kernel<EPI_UP>, pair::smem_bytes<EPI_UP>())) !=
                cudaSuccess ||
            (e = allow_smem(pair::mx4_gemm_2sm_kernel<EPI_DOWN>, pair::smem_bytes<EPI_DOWN>())) !=
                cudaSuccess ||
            (e = allow_smem(pair::mx4_down_res_kernel, 227 * 1024)) != cudaSuccess)
            return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        cluster_config(&cfg, attr, sms / 2, pair::smem_bytes<EPI_UP>(), nullptr);
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&n, pair::mx4_gemm_2sm_kernel<EPI_UP>, &cfg)) !=
            cudaSuccess)
            return e;
        di.pair_clusters = n > 0 ? n : 1;
        di.sms = sms;
    }
    *out = &di;
    return cudaSuccess;
}

// rank-2 map of a scale buffer (4-byte elements, boxes of 1024 bytes x `rows` tile rows)
static cudaError_t scale_map(CUtensorMap *map, const void *base, uint64_t tk, uint64_t tile_rows,
                             uint32_t rows)
{
    cudaError_t err;
    EncodeTiledFn enc = get_encoder(&err);
    if (enc == nullptr)
        return err != cudaSuccess ? err : cudaErrorSymbolNotFound;
    const cuuint64_t gd[2] = {tk * (kMx4Tile / 4), tile_rows}, gs[1] = {tk * kMx4Tile};
    const cuuint32_t bx[2] = {256, rows}, es[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), gd, gs, bx,
                           es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Which kernel and tile width.  The 1-SM kernel is bound by the 128-byte rows that a stage
// copies, so its cost is waves (tiles over the SMs) x those rows: A's of an average tile in
// boxes of 32, and B's.  A wave of the pair kernels and their longer start cost as much as the
// rows below, fitted to times at 1 to 64 experts, 2 to 12000 rows and 1 to 16 stages.  Row
// tiles are estimated for T*k rows spread evenly over the experts; each ragged end adds half a
// tile.  Measured (d 4096, m 1376, us; 192 / 128 / pair):
//   UP,   8 experts:  16 rows 11 / 13 / 18; 1024 rows 18 / 16 / 19; 2048 rows 21 / 22 / 20;
//                     8192 rows 53 / 65 / 42
//   UP,   1 expert:   200 rows 10 / 8.9 / 11; 1536 rows 17 / 16 / 12
//   DOWN, 8 experts:  406 rows 10 / 8.6 / 12; 2048 rows 17 / 20 / 18; 8192 rows 49 / 52 / 33
// Tiles of 64 columns won where they alone filled one wave, by up to 0.5 us in a product, and
// lost it in the FFN, where DOWN's loads begin on the SMs that UP leaves free (1 token 13.3 us
// with both at 64, 12.2 at 128).
struct Choice {
    bool two;
    int bn;
};
static Choice choose(const DevInfo &di, int64_t rows, int E, int N, int num_kb, bool resident)
{
    const int64_t hit = rows < E ? rows : E;
    auto row_tiles = [&](int bm) {
        const int64_t t = (2 * rows + (int64_t)bm * (hit - 1) + 2 * bm - 1) / (2 * bm);
        return t > hit ? t : hit;
    };
    const int64_t avg = (rows + hit - 1) / hit;
    const int a_rows = avg >= BM ? BM : ((int)avg + kABox - 1) / kABox * kABox;
    const int64_t pairs = row_tiles(2 * BM) * ((N + pair::BN - 1) / pair::BN);
    Choice c = {true, 0};
    const int start = resident ? 23000 / (15 * num_kb + 38) : 2400 / num_kb;
    const int wave = resident ? 250 + 170 / num_kb : 280;
    int64_t best = (pairs + di.pair_clusters - 1) / di.pair_clusters * wave + start;
    for (int w : {192, 128}) {
        const int64_t tiles = row_tiles(BM) * ((N + w - 1) / w);
        const int64_t cost = (tiles + di.sms - 1) / di.sms * (a_rows + w);
        if (cost < best) {
            best = cost;
            c = {false, w};
        }
    }
    return c;
}

template <int EPI, int BN>
static cudaError_t launch_1sm(const DevInfo &di, const CUtensorMap &ta, const CUtensorMap &tb,
                              const CUtensorMap &to, const GemmArgs &args, cudaStream_t s)
{
    return launch_pdl(mx4_gemm_kernel<EPI, BN>, dim3(di.sms), dim3(NUM_THREADS),
                      Geo<EPI, BN>::SMEM, s, ta, tb, to, args);
}

template <int EPI>
static cudaError_t launch_gemm(const void *A, const void *B, const GemmArgs &args, cudaStream_t s)
{
    const int64_t rows = args.rows;
    DevInfo *di = nullptr;
    cudaError_t e = prepare_device(&di);
    if (e != cudaSuccess)
        return e;
    const int num_kb = (args.K32 + BKC - 1) / BKC;
    const bool resident = EPI == EPI_DOWN && num_kb <= pair::kResKb;
    const Choice ch = choose(*di, rows, args.E, args.N, num_kb, resident);
    const bool two = ch.two;
    const int bn = ch.bn;
    // code rows as 2-byte elements (four codes each): the maps only copy
    const uint64_t kel = (uint64_t)args.K32 / 4, pitch = (uint64_t)args.K32 / 2;
    CUtensorMap ta, tb, to = {};
    const uint64_t da[2] = {kel, (uint64_t)rows}, sa[1] = {pitch};
    const uint64_t db[3] = {kel, (uint64_t)args.N, (uint64_t)args.E};
    const uint64_t sb[2] = {pitch, pitch * args.N};
    const uint32_t ba[2] = {BKB / 2, (uint32_t)(two ? BM : kABox)}, bb[3] = {BKB / 2, (uint32_t)(two ? pair::BNH : bn), 1};
    if ((e = make_map(&ta, A, 2, da, sa, ba)) != cudaSuccess ||
        (e = make_map(&tb, B, 3, db, sb, bb)) != cudaSuccess)
        return e;
    if (EPI == EPI_DOWN) {  // output boxes of 32 columns x 32 rows
        const uint64_t dout[2] = {(uint64_t)args.n_valid, (uint64_t)rows}, sout[1] = {(uint64_t)args.ld * 2};
        const uint32_t bout[2] = {32, 32};
        if ((e = make_map(&to, args.out, 2, dout, sout, bout, CU_TENSOR_MAP_SWIZZLE_64B)) != cudaSuccess)
            return e;
    }
    if (!two) {
        if (bn == 128)
            return launch_1sm<EPI, 128>(*di, ta, tb, to, args, s);
        return launch_1sm<EPI, 192>(*di, ta, tb, to, args, s);
    }
    CUtensorMap tsa, tsb;
    const uint64_t tk = (args.K32 + 127) / 128;
    if ((e = scale_map(&tsa, args.a_s, tk, (uint64_t)mx4_row_tiles(rows, args.E), 1)) != cudaSuccess ||
        (e = scale_map(&tsb, args.b_s, tk, (uint64_t)args.E * ((args.N + 127) / 128), 2)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (resident) {
        cluster_config(&cfg, attr, di->pair_clusters, pair::res_smem(num_kb), s);
        return cudaLaunchKernelEx(&cfg, pair::mx4_down_res_kernel, ta, tb, tsa, tsb, to, args,
                                  pair::res_stages(num_kb));
    }
    cluster_config(&cfg, attr, di->pair_clusters, pair::smem_bytes<EPI>(), s);
    const int band_rows = gemm_band_rows();
    const int band = band_rows <= 0 ? 0 : (band_rows + 2 * BM - 1) / (2 * BM);
    return cudaLaunchKernelEx(&cfg, pair::mx4_gemm_2sm_kernel<EPI>, ta, tb, tsa, tsb, to, args, band);
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
    a.rows = p->T * p->k;
    a.N = 2 * round_up(p->m, 16);
    a.K32 = p->d;
    a.n_valid = p->m;
    a.ld = mx4_k32(p->m) / 2;
    a.status = status;
    a.wait_ns = wait_limit_ns();
    count_launch();
    return mxg::launch_gemm<mxg::EPI_UP>(xq, W13q, a, s);
}

cudaError_t launch_mx4_down(const moe_params_t *p, const void *hq, const void *hs,
                            const int32_t *offsets, const void *W2q, const void *W2s, void *out,
                            bool after_up, int32_t *status, cudaStream_t s)
{
    mxg::GemmArgs a = {};
    a.a_s = (const uint8_t *)hs;
    a.b_s = (const uint8_t *)W2s;
    a.offsets = offsets;
    a.out = out;
    a.E = p->E;
    a.rows = p->T * p->k;
    a.N = p->d;
    a.K32 = mx4_k32(p->m);
    a.n_valid = p->d;
    a.ld = p->d;
    a.after_up = after_up;
    a.status = status;
    a.wait_ns = wait_limit_ns();
    count_launch();
    return mxg::launch_gemm<mxg::EPI_DOWN>(hq, W2q, a, s);
}

}  // namespace moe
