// mx4_few.cu -- the whole layer for 1..16 tokens on mx4 expert weights and bf16
// activations, in one cooperative launch (moe_forward_mx4, MOE_MX4_ACT_BF16).
// Router: "Llama 3 Meets MoE: Efficient Upcycling", section 3 "核心公式" (section 5 for the
// Mixtral and ST types); capacity: its "容量因子"; SwiGLU expert: "LLaMA-MoE v2", code
// sample, class Expert; statistics: "LLaMA-MoE v2", section "门控机制设计".
//
// The selected experts' weights (0.53 bytes each) are all it has to read; the chain routing ->
// GEMM 1 -> grid barrier -> GEMM 2 takes longer, and no unit is full on the way (8 tokens: issue
// slots 43 %, integer pipe 39 %, tensor pipe 12 %, DRAM 19 %).  Its 4 warps a scheduler wait: of the
// 9.2 cycles between two instructions of a warp 2.2 are for the next instruction to be fetched (3.3
// of 11 at 1 token), 1.2 for the result of the last, 1.0 for the pipes, 0.9 at barriers (2.0), 0.6
// for global loads.  Measured (d 4096, graph replays, weights in L2 / after 512 MB of other reads):
// 1 token of 8 experts x 1376, top 2, 18.4 / 24.7 us (18.2 MB), 8 tokens 30.7 to 34 / 41 to 44 us
// (65 MB), 16 tokens of 16 x 688, top 4, 53.3 to 57 / 67 us (71 MB); ranges over inputs.
//
//   routing   every CTA computes all logits (mma.sync on bf16), gates and tables: x and W_g
//             are some ten KB and no CTA waits for another.
//   GEMM 1    the selected experts' neurons are split evenly over the CTAs; an item is 8
//             neurons of one expert: their W1 rows are A rows 0..7 of mma.sync m16n8k16,
//             their W3 rows A rows 8..15.  B is all of the batch's tokens, whatever the
//             expert (8 columns cost what one does): a warp's slice of 256 columns stays in
//             its registers for every item, and the epilogue keeps the routed tokens.
//   GEMM 2    after a grid barrier (h complete): each CTA owns a strip of at most 32 output
//             columns.  Column t of B is token t's row of h in the expert at hand; a warp
//             walks over (expert, 256 columns of h) and adds gate weight * product to the
//             same sums throughout, so one reduction ends in y.
//
// The product.  e2m1 values are exact in f16 (one conversion per pair), so A is the codes
// themselves; B is the bf16 activations scaled by a power of two per 128 columns to a maximum
// in [2^13, 2^14): exact in f16 down to 2^-27 of that maximum, off by less than 2^-38 of it
// below.  The two products of a 32-column block accumulate in f32 and are added to the sum
// times the block's scale, so the weights' scales may lie any distance apart.  A lane's
// k indexes are 8 consecutive columns, for A and B alike (the order of k inside a product
// is free).
//
// Weights stream through two stages of 32 rows x 256 columns with their 64 scale words, which
// each warp fills for itself with cp.async, one stage ahead and across items: no barrier
// between loads and products but __syncwarp.  The loop's work is the conversions (integer pipe)
// and the load unit's lines and wavefronts: B stays in registers (it never passes through
// shared memory), a copy instruction covers whole 128-byte lines of 4 rows, and
// rows are enumerated in the order of the scale tiles -- 4 rows that lie 32 apart share 16
// bytes of scales -- so that one copy instruction brings all scales of a stage.  Partial sums
// meet in shared memory in warp order, so results do not depend on timing.
#include <mutex>
#include <type_traits>

#include "gate.cuh"
#include "mx4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace few {

using tc::smem_u32;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kChunkBytes = 16 * 64 + 64;     // 16 rows x 128 columns: codes, scale words
constexpr int kSlice = 256;                   // columns of a stage
constexpr int kStageBytes = 4 * kChunkBytes;  // 32 rows x 256 columns: [16 rows][128 columns]
constexpr int kRingBytes = kWarps * 2 * kStageBytes;
constexpr int kWindow1 = kWarps * kSlice;     // columns of x at a time
constexpr int kStrip = 32;                    // GEMM 2: output columns at a time
constexpr int kMaxRows = MOE_MX4_FEW_TOKENS * MOE_MAX_TOPK;
constexpr int kMaxE = 32;
constexpr int kRegion = 72 * 1024;            // the warps' sums
constexpr int kSmem = kRegion + kRingBytes;   // dynamic; beside it the tables below
constexpr int kItems = 512;                   // GEMM 1's items at a time

// Routing and work tables of a CTA (static shared memory)
struct Tables {
    uint32_t mask[kMaxE];  // tokens that chose an expert
    int32_t off[kMaxE + 1], sel[kMaxE];
    int32_t idx[kMaxRows], slot[kMaxRows], rtok[kMaxRows];
    int8_t map[kMaxE * MOE_MX4_FEW_TOKENS];  // row of (expert, token), -1 none
    float w[kMaxRows], rw[kMaxRows];
    float lg[MOE_MX4_FEW_TOKENS * 32], prob[MOE_MX4_FEW_TOKENS * kMaxE], gw[MOE_MX4_FEW_TOKENS * kMaxE];
    int32_t items[kItems];
    int abort;
};
static_assert(kSmem + sizeof(Tables) <= 227 * 1024, "shared memory of a CTA");
static_assert(kMaxE * MOE_MX4_FEW_TOKENS == kThreads, "one thread clears an entry of the map");
static_assert(kMaxRows <= 128 && kMaxRows <= kThreads - 32, "rows in 8 bits; one thread a row");

struct Args {
    const bf16 *x, *Wg, *Wn;
    const float *noise, *bias;
    const uint8_t *W13q, *W13s, *W2q, *W2s;
    bf16 *h, *y;
    float *loss, *importance, *f, *P, *probs_sum, *w;
    int32_t *counts, *idx, *row_token, *slot_row, *kept, *offsets;
    int32_t *status;
    unsigned long long *gbar;  // arrivals at the grid barrier, ever
    uint64_t wait_ns;
    float lambda, scale;
    int T, d, m, E, k, C, router_type;
    int tk1, tk2;      // tiles of a scale tile row of W13, W2
    int64_t w13_codes, w13_scales, w2_codes, w2_scales;  // bytes of one expert
};

// 16 bytes to shared memory; zeros where `on` is false (nothing is read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait()  // all but the newest N groups
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ unsigned long long ld_acquire_u64(const unsigned long long *p)
{
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&b)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same with C = 0
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// --------------------------------------------------------------------- work items
// GEMM 1 works on quads of neurons (4 that share 16 bytes of scales), 16 quads per 64
// neurons: quad q is neurons 64 (q / 16) + q % 16 + 16 i.  A CTA takes quads [lo, hi) of
// the selected experts' (expert-major), four per item, items inside one expert.
struct UpItems {
    int lo, hi, per;       // per: quads of an expert (a multiple of 16)
    int is0, at0, first;   // the first expert, the first quad in it, its items
    __device__ __forceinline__ UpItems(int nsel, int m)
    {
        per = (m + 63) / 64 * 16;
        const uint32_t all = (uint32_t)(nsel * per);  // at most 2^23, times the grid below 2^32
        lo = (int)(blockIdx.x * all / gridDim.x);
        hi = (int)((blockIdx.x + 1) * all / gridDim.x);
        is0 = lo / per;
        at0 = lo - is0 * per;
        first = (min(hi - lo, per - at0) + 3) / 4;
    }
    __device__ __forceinline__ int count() const
    {
        if (hi <= lo)
            return 0;
        const int rest = hi - lo - min(hi - lo, per - at0);
        return first + rest / per * (per / 4) + (rest % per + 3) / 4;
    }
    // item i: its expert (position among the selected), first quad, quads (1..4)
    __device__ __forceinline__ void get(int i, int &is, int &q, int &n) const
    {
        is = is0;
        q = at0 + 4 * i;
        if (i >= first) {
            i -= first;
            for (++is; i >= per / 4; ++is)
                i -= per / 4;
            q = 4 * i;
        }
        n = min(4, min(hi - is * per - q, per - q));
    }
};
// neuron s (0..15) of an item that starts at quad q
__device__ __forceinline__ int up_neuron(int q, int s)
{
    const int qq = q + s / 4;
    return qq / 16 * 64 + qq % 16 + 16 * (s % 4);
}

// GEMM 2 works on quads of output columns, 32 quads per 128 columns: quad q is columns
// 128 (q / 32) + q % 32 + 32 i.  A CTA takes quads [lo, hi), eight per strip; the s-th column
// counted from quad q on:
__device__ __forceinline__ int down_column(int q, int s)
{
    const int qq = q + s / 4;
    return qq / 32 * 128 + qq % 32 + 32 * (s % 4);
}

// --------------------------------------------------------------------- weight rings
// GEMM 1's items, at most kItems at a time, as a table in shared memory: expert, quads and
// first quad packed into a word (the divisions behind them are made once per item).
__device__ __forceinline__ int32_t item_pack(int e, int q, int n) { return e | n << 5 | q << 8; }
__device__ __forceinline__ int item_expert(int32_t v) { return v & 31; }
__device__ __forceinline__ int item_quads(int32_t v) { return v >> 5 & 7; }
__device__ __forceinline__ int item_first(int32_t v) { return v >> 8; }

// How GEMM 1 is shared out: 2^kshift warps (a group) hold the slices of a window of x, the
// groups take the items of a batch in turn.
struct UpPlan {
    int n, batch, kshift, n_win;  // n: items in the table; batch: items between reductions
    __device__ __forceinline__ UpPlan(int d, int nb)
    {
        n = 0;
        n_win = (d + kWindow1 - 1) / kWindow1;
        const int slices = (min(d, kWindow1) + kSlice - 1) / kSlice;
        kshift = 32 - __clz(slices - 1);  // 0 for one slice
        batch = kRegion / (nb * 1024) >> kshift;
    }
    __device__ __forceinline__ int group() const { return (int)(threadIdx.x >> 5) >> kshift; }
    __device__ __forceinline__ int groups() const { return kWarps >> kshift; }
    // first column of this warp's slice of window w
    __device__ __forceinline__ int column(int w) const
    {
        return w * kWindow1 + ((int)(threadIdx.x >> 5) & ((1 << kshift) - 1)) * kSlice;
    }
};
// A warp's way through a table: batches of items, windows, the group's items.
struct UpWalk {
    int b0, w, i, end;  // end: of the batch
    __device__ __forceinline__ UpWalk(const UpPlan &p) : b0(0), w(0), i(p.group()), end(min(p.batch, p.n))
    {
        skip(p);
    }
    __device__ __forceinline__ bool on(const UpPlan &p) const { return b0 < p.n; }
    __device__ __forceinline__ void next(const UpPlan &p)
    {
        i += p.groups();
        skip(p);
    }
    __device__ __forceinline__ void skip(const UpPlan &p)
    {
        while (__builtin_expect(i >= end && b0 < p.n, 0)) {
            if (++w == p.n_win) {
                w = 0;
                b0 = end;
                end = min(b0 + p.batch, p.n);
            }
            i = b0 + p.group();
        }
    }
};

// A lane's place in a stage.  A copy instruction brings 128-byte lines (256 columns) of the 4
// rows of a quad: lane l has row l / 8 of it and 16-byte piece l % 8, which belongs to 128-
// column chunk l / 4 % 2.  Rows lie 64 bytes apart in a chunk, their 4 pieces swizzled by
// (row / 2) % 4; quads 2 j and 2 j + 1 of 8 rows differ in that swizzle.
struct Place {
    uint32_t quad[2];
    __device__ __forceinline__ Place()
    {
        const int lane = threadIdx.x & 31, row = lane >> 3, piece = lane & 3;
        const uint32_t u = (uint32_t)((lane >> 2 & 1) * kChunkBytes + row * 64);
        quad[0] = u + (uint32_t)((piece ^ (row >> 1)) << 4);
        quad[1] = u + (uint32_t)(256 + ((piece ^ (2 + (row >> 1))) << 4));
    }
    // quad i of a 32-row stage: chunks [16 rows][128 columns], 4 quads of 4 rows each
    __device__ __forceinline__ uint32_t at(int i) const
    {
        return (uint32_t)((i >> 2) * 2 * kChunkBytes + (i >> 1 & 1) * 512) + quad[i & 1];
    }
};

// Fills a stage of GEMM 1 (one group of copies): the item's 16 neurons, W1 rows of the first 8
// and their W3 rows, then the other 8, x the 256 columns from col on.  Quad qq is W13 rows
// 128 (qq / 16) + qq % 16 + 32 i, its W3 rows 16 further; their scale words are 16 bytes at
// 16 (qq % 16 [+ 16]) of tile qq / 16.  Rows past the expert's and columns past d become zeros.
__device__ __forceinline__ void up_fill(const Args &a, int32_t item, int col, uint32_t st,
                                        const Place &place)
{
    const int lane = threadIdx.x & 31, r = lane >> 3;
    const int e = item_expert(item), n = item_quads(item), q = item_first(item);
    const int half = a.d >> 1, at = (col >> 1) + (lane & 7) * 16;
    const uint8_t *ce = a.W13q + e * a.w13_codes + (int64_t)(32 * r) * half + at;
    const bool in = at < half;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int qq = q + j;
        const bool on = in && j < n && (qq >> 4) * 64 + (qq & 15) + 16 * r < a.m;
        const uint8_t *s0 = ce + (int64_t)((qq >> 4) * 128 + (qq & 15)) * half;
        cp16(st + place.at((j >> 1) * 4 + (j & 1)), s0, on);
        cp16(st + place.at((j >> 1) * 4 + 2 + (j & 1)), s0 + 16 * half, on);
    }
    // scales: lane = (chunk, W1 or W3, quad)
    if (lane < 16) {
        const int j = lane & 3, up = lane >> 2 & 1, u = lane >> 3, qq = q + j, ch = (col >> 7) + u;
        cp16(st + (uint32_t)((2 * (j >> 1) + u) * kChunkBytes + 1024 + up * 32 + (j & 1) * 16),
             a.W13s + e * a.w13_scales + ((int64_t)((qq >> 4) * a.tk1) + ch) * kMx4Tile +
                 ((qq & 15) + 16 * up) * 16,
             j < n && ch < a.tk1);
    }
    cp_commit();
}

// How GEMM 2 is shared out: the (selected expert, 256 columns of h) pairs go round the warps.
struct DownPlan {
    int lo, hi, strips, nsel, units;  // units: of an expert
    __device__ __forceinline__ DownPlan(const Args &a, int sel)
    {
        const uint32_t all = (uint32_t)((a.d + 127) / 128 * 32);
        lo = (int)(blockIdx.x * all / gridDim.x);
        hi = (int)((blockIdx.x + 1) * all / gridDim.x);
        strips = (4 * (hi - lo) + kStrip - 1) / kStrip;
        nsel = sel;
        units = (a.m + kSlice - 1) / kSlice;
    }
};
// A warp's way: strips, its pairs (is: expert among the selected, u: unit).
struct DownWalk {
    int strip, is, u;
    __device__ __forceinline__ DownWalk(const DownPlan &p)
    {
        strip = p.nsel == 0 ? p.strips : 0;
        first(p);
    }
    __device__ __forceinline__ bool on(const DownPlan &p) const { return strip < p.strips; }
    __device__ __forceinline__ void first(const DownPlan &p)
    {
        is = 0;
        u = (int)threadIdx.x >> 5;
        wrap(p);
        if (is >= p.nsel)  // no pair for this warp
            strip = p.strips;
    }
    __device__ __forceinline__ void wrap(const DownPlan &p)
    {
        while (u >= p.units) {
            u -= p.units;
            ++is;
        }
    }
    __device__ __forceinline__ void next(const DownPlan &p)
    {
        u += kWarps;
        wrap(p);
        if (__builtin_expect(is >= p.nsel, 0)) {
            ++strip;
            first(p);
        }
    }
};

// Fills a stage of GEMM 2 (one group of copies): the strip's 8 quads of W2 rows of expert e x
// the 256 columns from col on; rows past the strip and columns past K32 become zeros.
__device__ __forceinline__ void down_fill(const Args &a, const DownPlan &p, int strip, int e, int col,
                                          uint32_t st, const Place &place)
{
    const int lane = threadIdx.x & 31, r = lane >> 3, q = p.lo + 8 * strip, n = p.hi - q;
    const int half = mx4_k32(a.m) >> 1, at = (col >> 1) + (lane & 7) * 16;
    const uint8_t *ce = a.W2q + e * a.w2_codes + (int64_t)(32 * r) * half + at;
    const bool in = at < half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int qq = q + i, row = (qq >> 5) * 128 + (qq & 31);
        cp16(st + place.at(i), ce + (int64_t)row * half, in && i < n && row + 32 * r < a.d);
    }
    if (lane < 16) {  // scales: lane = (chunk, quad)
        const int i = lane & 7, u = lane >> 3, qq = q + i, ch = (col >> 7) + u;
        cp16(st + (uint32_t)((2 * (i >> 2) + u) * kChunkBytes + 1024 + (i & 3) * 16),
             a.W2s + e * a.w2_scales + ((int64_t)((qq >> 5) * a.tk2) + ch) * kMx4Tile + (qq & 31) * 16,
             i < n && (qq >> 5) * 128 < a.d && ch < a.tk2);
    }
    cp_commit();
}

// --------------------------------------------------------------------- activations
// The power of two that takes a maximum with the bf16 magnitude bits `top` into [2^13, 2^14):
// 2^(13 - floor(log2(max))), exponent field 127 + 13 - (E - 127), at most 254.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) { return min(267u - (top >> 7), 254u); }

// largest magnitude bits of two bf16 values in each half of a word: max of the halves, apart
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t top_of(const uint4 &v)
{
    return max_halves(max_halves(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                      max_halves(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}

// 8 bf16 values times mul, as f16
__device__ __forceinline__ void to_half(uint4 &v, float mul)
{
    float f[8];
    bf16x8_to_f32(v, f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 hh = __floats2half2_rn(f[2 * i] * mul, f[2 * i + 1] * mul);
        o[i] = *reinterpret_cast<const uint32_t *>(&hh);
    }
    v = make_uint4(o[0], o[1], o[2], o[3]);
}

// B of a stage in registers, as stored: columns [col, col + 256) of the rows at src[nb] (this
// lane's row of each group of 8 tokens, nullptr: zeros), 8 columns of each of the 8 blocks;
// columns from `limit` on are zeros.  CG: rows that other SMs wrote in this launch.
template <int NB, bool CG>
__device__ __forceinline__ void load_b(const bf16 *const (&src)[NB], int col, int limit,
                                       uint4 (&xb)[NB][8])
{
    const int c = threadIdx.x & 3;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const int at = col + 32 * b + 8 * c;
            xb[nb][b] = make_uint4(0, 0, 0, 0);
            if (src[nb] != nullptr && at < limit)
                xb[nb][b] = CG ? __ldcg(reinterpret_cast<const uint4 *>(src[nb] + at)) : ld_nc(src[nb] + at);
        }
}

// Turns them into scaled f16; inv[nb][u][j]: weight of token 2c + j's row (w[nb] of the lane
// that holds it) times the inverse of its scale in chunk u.  limit: as above (the 8 columns
// around it come with whatever lies behind them).
template <int NB>
__device__ __forceinline__ void scale_b(uint4 (&xb)[NB][8], int col, int limit, const float (&w)[NB],
                                        float (&inv)[NB][2][2])
{
    const int lane = threadIdx.x & 31, c = lane & 3;
    if (col + kSlice > limit && (limit & 7) != 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const int n = limit - (col + 32 * b + 8 * c);  // columns that exist
                if (n > 0 && n < 8) {
                    uint32_t v[4] = {xb[nb][b].x, xb[nb][b].y, xb[nb][b].z, xb[nb][b].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = 2 * i + 1 < n ? v[i] : (2 * i < n ? v[i] & 0xffffu : 0u);
                    xb[nb][b] = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                top = max_halves(top, top_of(xb[nb][4 * u + b]));
            top = max_halves(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max_halves(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t field = scale_field(max(top & 0xffffu, top >> 16));
#pragma unroll
            for (int b = 0; b < 4; ++b)
                to_half(xb[nb][4 * u + b], __uint_as_float(field << 23));
            const float r = mx4_scale(254u - field) * w[nb];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                inv[nb][u][j] = __shfl_sync(0xffffffffu, r, (2 * c + j) * 4);
        }
}

// 2^s of the four bytes of a scale word (0: 2^-127, 255: NaN, as the conversion has them)
__device__ __forceinline__ void word_scales(uint32_t w, float (&s)[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    s[0] = __uint_as_float(lo << 16);
    s[1] = __uint_as_float(lo & 0xffff0000u);
    s[2] = __uint_as_float(hi << 16);
    s[3] = __uint_as_float(hi & 0xffff0000u);
}

// sum = A chunk * B: the chunk's 16 rows (at `st`, this lane's words of row g at off[b])
// against this lane's B fragments x[nb][b].
template <int NB, class X>
__device__ __forceinline__ void chunk_mma(float (&sum)[NB][4], uint32_t st, const uint32_t (&off)[4],
                                          const X &x, int g)
{
    float s0[4], s1[4];
    word_scales(lds32(st + 1024 + g * 4), s0);
    word_scales(lds32(st + 1056 + g * 4), s1);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t a0[4], a1[4];
        mx4_halves8(lds32(st + off[b]), a0);
        mx4_halves8(lds32(st + off[b] + 512), a1);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint4 v = x(nb, b);
            float t[4];
            mma_f16_first(t, a0[0], a1[0], a0[1], a1[1], v.x, v.y);
            mma_f16(t, a0[2], a1[2], a0[3], a1[3], v.z, v.w);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float f = q < 2 ? s0[b] : s1[b];
                sum[nb][q] = b == 0 ? t[q] * f : fmaf(t[q], f, sum[nb][q]);
            }
        }
    }
}

// --------------------------------------------------------------------- the router
// The logits lg [T][nout] of all tokens.  A group's warps have the slices of a window of x in
// registers already (x, of window 0; left holding the last window's); the groups share a
// slice's 32-column steps, step s to group s % groups.  The warp's rows of [W_g | W_noise] pass
// through its own `stage` bytes, and the warps' sums (`part`) are added in warp order.
template <int NB>
__device__ __forceinline__ void router_logits(const Args &a, const UpPlan &p, uint4 (&x)[NB][8],
                                              char *stage, int stage_bytes, float *part, float *lg)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int E = a.E, T = a.T, d = a.d, nout = a.Wn != nullptr ? 2 * E : E;
    const int NT = (nout + 7) / 8, NP = NT * 8;
    const int room = stage_bytes / (64 * NP), grp = p.group(), gshift = 4 - p.kshift;
    const uint32_t sb = smem_u32(stage);
    float acc[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            acc[nt][q] = 0.f;
#pragma unroll 1
    for (int w = 0; w < p.n_win; ++w) {
        const int col = p.column(w), steps = min(8, (d - col + 31) >> 5);  // none past d
        if (w > 0) {
            const bf16 *src[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                src[nb] = nb * 8 + g < T ? a.x + (int64_t)(nb * 8 + g) * d : nullptr;
            load_b<NB, false>(src, col, d, x);
        }
        const int mine = (steps - grp + (1 << gshift) - 1) >> gshift;  // steps of this warp
#pragma unroll 1
        for (int k0 = 0; k0 < mine; k0 += room) {
            const int n = min(room, mine - k0);
            const bf16 *wg = a.Wg + (int64_t)col * E, *wn = a.Wn + (int64_t)col * E;
            __syncwarp();
            if ((E & 7) == 0) {  // rows of whole 16-byte pieces
#pragma unroll 4
                for (int i = lane; i < n * 32 * NT; i += 32) {
                    const int k = NT == 1 ? i : i / NT, o = (i - k * NT) * 8;
                    const int row = (grp + ((k0 + (k >> 5)) << gshift)) * 32 + (k & 31);
                    cp16(sb + i * 16, o < E ? wg + (int64_t)row * E + o : wn + (int64_t)row * E + o - E, true);
                }
                cp_commit();
                cp_wait<0>();
            } else {
                const bf16 zero = __float2bfloat16_rn(0.f);
#pragma unroll 8
                for (int i = lane; i < n * 32 * NP; i += 32) {
                    const int k = i / NP, o = i - k * NP;
                    const int row = (grp + ((k0 + (k >> 5)) << gshift)) * 32 + (k & 31);
                    reinterpret_cast<bf16 *>(stage)[i] =
                        o < E ? wg[(int64_t)row * E + o]
                              : (o < nout ? wn[(int64_t)row * E + o - E] : zero);
                }
            }
            __syncwarp();
#pragma unroll
            for (int b = 0; b < 8; ++b) {  // unrolled: x stays in registers
                const int k = (b >> gshift) - k0;
                if ((b & ((1 << gshift) - 1)) != grp || k < 0 || k >= n || b >= steps)
                    continue;
                // A: 8 consecutive columns of token rows g, g + 8.  B of the two products:
                // columns 8c + {0,1 | 2,3} and 8c + {4,5 | 6,7}
                const uint4 x0 = x[0][b], x1 = NB == 2 ? x[NB - 1][b] : make_uint4(0, 0, 0, 0);
                const int i = lane & 7, kk = k * 32 + 8 * (i >> 1) + (i & 1) + 2 * (lane >> 3);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    if (nt >= NT)
                        break;
                    uint32_t f[4];
                    ldsm_x4_trans(sb + (uint32_t)(kk * NP * 2 + nt * 16), f);
                    mma_bf16_16816(acc[nt], x0.x, x1.x, x0.y, x1.y, f[0], f[1]);
                    mma_bf16_16816(acc[nt], x0.z, x1.z, x0.w, x1.w, f[2], f[3]);
                }
            }
        }
    }
    float *pw = part + (size_t)warp * T * NP;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        const int o = nt * 8 + 2 * c;
        if (nt < NT && g < T) {
            pw[g * NP + o] = acc[nt][0];
            pw[g * NP + o + 1] = acc[nt][1];
        }
        if (nt < NT && NB == 2 && g + 8 < T) {
            pw[(g + 8) * NP + o] = acc[nt][2];
            pw[(g + 8) * NP + o + 1] = acc[nt][3];
        }
    }
    __syncthreads();
    if (warp < T && lane < nout) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            sum += part[((size_t)w * T + warp) * NP + lane];
        lg[warp * nout + lane] = sum;
    }
    __syncwarp();  // the gate of token t is warp t's
}

// --------------------------------------------------------------------- the kernel
template <int NB>
__global__ void __launch_bounds__(kThreads, 1) mx4_few_kernel(const __grid_constant__ Args a)
{
    extern __shared__ __align__(128) char sm[];
    __shared__ Tables tab;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int T = a.T, E = a.E, k = a.k, d = a.d, m = a.m;
    char *region = sm;  // the router's sums, GEMM 1's, then the rows of h
    char *my_ring = sm + kRegion + warp * 2 * kStageBytes;
    const uint32_t ring_s = smem_u32(my_ring);
    // x first: this warp's slice of window 0, as it lies
    UpPlan plan(d, NB);
    const bf16 *xsrc[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
        xsrc[nb] = nb * 8 + g < T ? a.x + (int64_t)(nb * 8 + g) * d : nullptr;
    uint4 xb[NB][8];
    load_b<NB, false>(xsrc, plan.column(0), d, xb);
    // The grid barrier counts arrivals for ever, gridDim.x a launch: this launch's are complete
    // when the count reaches the next multiple.
    unsigned long long target = 0;
    if (threadIdx.x == kThreads - 1) {
        tab.abort = 0;
        const unsigned long long n = ld_acquire_u64(a.gbar);
        target = (n / gridDim.x + 1) * gridDim.x;
    }
    tab.map[threadIdx.x] = -1;
    if (threadIdx.x < kMaxE)
        tab.mask[threadIdx.x] = 0;

    // ---- router
    const int nout = a.Wn != nullptr ? 2 * E : E;
    float *part = reinterpret_cast<float *>(region);
    router_logits<NB>(a, plan, xb, my_ring, 2 * kStageBytes, part, tab.lg);
    if (warp < T)
        gate_token_warp(tab.lg + warp * nout, E, k, a.Wn != nullptr ? 1 : 0,
                        a.noise + (a.noise != nullptr ? (size_t)warp * E : 0), a.bias, a.router_type,
                        tab.idx + warp * k, tab.w + warp * k, tab.prob + warp * E, tab.gw + warp * E,
                        a.status);
    __syncwarp();
    if (warp < T && lane < k && tab.idx[warp * k + lane] >= 0)
        atomicOr(&tab.mask[tab.idx[warp * k + lane]], 1u << warp);
    __syncthreads();
    // ---- dispatch tables (stable by token, assignments past the capacity dropped).  tab.mask[e]
    // has a bit for each token that chose expert e, so a row's rank is a population count and
    // every warp makes the experts' tables for itself (all write the same values).
    int nsel;
    {
        const uint32_t chosen = lane < E ? tab.mask[lane] : 0u;
        const int cnt = __popc(chosen), kept = a.C < 0 ? cnt : min(cnt, a.C);
        int off = kept;  // inclusive prefix sum
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, off, o);
            off += lane >= o ? u : 0;
        }
        const uint32_t used = __ballot_sync(0xffffffffu, kept > 0);
        nsel = __popc(used);
        if (lane < E) {
            tab.off[lane + 1] = off;
            if (lane == 0)
                tab.off[0] = 0;
            if (kept > 0)
                tab.sel[__popc(used & ((1u << lane) - 1))] = lane;
        }
        // warp t: the rows of token t
        const int e = warp < T && lane < k ? tab.idx[warp * k + lane] : -1;
        const int first = __shfl_sync(0xffffffffu, off - kept, max(e, 0));
        const int room = __shfl_sync(0xffffffffu, kept, max(e, 0));
        if (warp < T && lane < k) {
            const int rank = e < 0 ? 0 : __popc(tab.mask[e] & ((1u << warp) - 1));
            const int row = e >= 0 && rank < room ? first + rank : -1;
            tab.slot[warp * k + lane] = row;
            if (row >= 0) {
                tab.rtok[row] = warp;
                tab.rw[row] = tab.w[warp * k + lane];
                tab.map[e * MOE_MX4_FEW_TOKENS + warp] = (int8_t)row;
            }
        }
        __syncwarp();
    }
    const int R = tab.off[E], m8 = round_up(m, 8);
    const Place place;
    uint32_t a_off[4];  // this lane's words of A row g in a chunk
#pragma unroll
    for (int b = 0; b < 4; ++b)
        a_off[b] = (uint32_t)(g * 64 + ((b ^ ((g >> 1) & 3)) << 4) + c * 4);

    // ---- GEMM 1
    {
        const UpItems up(nsel, m);
        const int n_up = up.count();
        float *sums = reinterpret_cast<float *>(region);
        // sums of an item: [slice][half][nb][lane] float4
        const int nks = 1 << plan.kshift, ks = warp & (nks - 1);
        float inv[NB][2][2], one[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            one[nb] = 1.f;
#pragma unroll 1
        for (int base = 0; base < n_up; base += kItems) {
            plan.n = min(kItems, n_up - base);
            if (base > 0)
                __syncthreads();  // the table's last use is over
            for (int j = lane; j < plan.n; j += 32) {  // every warp for itself, the same values
                int is, q, n;
                up.get(base + j, is, q, n);
                tab.items[j] = item_pack(tab.sel[is], q, n);
            }
            __syncwarp();
            UpWalk ld(plan);
            if (ld.on(plan)) {
                up_fill(a, tab.items[ld.i], plan.column(ld.w), ring_s, place);
                ld.next(plan);
            }
            uint32_t st = 0;
            if (plan.n_win == 1 && base == 0)
                scale_b<NB>(xb, plan.column(0), d, one, inv);
#pragma unroll 1
            for (int b0 = 0; b0 < plan.n; b0 += plan.batch) {
                const int b1 = min(b0 + plan.batch, plan.n);
#pragma unroll 1
                for (int w = 0; w < plan.n_win; ++w) {
                    if (plan.n_win > 1) {
                        load_b<NB, false>(xsrc, plan.column(w), d, xb);
                        scale_b<NB>(xb, plan.column(w), d, one, inv);
                    }
#pragma unroll 1
                    for (int i = b0 + plan.group(); i < b1; i += plan.groups()) {
                        __syncwarp();  // the other stage has been read
                        if (ld.on(plan)) {
                            up_fill(a, tab.items[ld.i], plan.column(ld.w), ring_s + (st ^ kStageBytes), place);
                            ld.next(plan);
                        } else {
                            cp_commit();
                        }
                        cp_wait<1>();
                        __syncwarp();
                        float4 *o = reinterpret_cast<float4 *>(sums) +
                                    (size_t)((((i - b0) << plan.kshift) + ks) * 2 * NB) * 32 + lane;
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            float acc[NB][4];
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                float sum[NB][4];
                                chunk_mma<NB>(sum, ring_s + st + (2 * h + u) * kChunkBytes, a_off,
                                              [&](int nb, int b) { return xb[nb][4 * u + b]; }, g);
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        const float f = inv[nb][u][q & 1];
                                        acc[nb][q] = u == 0 ? sum[nb][q] * f : fmaf(sum[nb][q], f, acc[nb][q]);
                                    }
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                float4 v = make_float4(acc[nb][0], acc[nb][1], acc[nb][2], acc[nb][3]);
                                if (w > 0) {
                                    const float4 p = o[nb * 32];
                                    v = make_float4(p.x + v.x, p.y + v.y, p.z + v.z, p.w + v.w);
                                }
                                o[nb * 32] = v;
                            }
                            o += NB * 32;
                        }
                        st ^= kStageBytes;
                    }
                }
                __syncthreads();
                // the slices' sums in order, SwiGLU, h of the routed tokens: one warp per item,
                // half and nb; lane (s, c) has gate and up of neuron s for tokens 2c, 2c + 1
#pragma unroll 1
                for (int j = warp; j < (b1 - b0) * 2 * NB; j += kWarps) {
                    const int i = j / (2 * NB), hb = j % (2 * NB);
                    const int32_t item = tab.items[b0 + i];
                    const float4 *r = reinterpret_cast<const float4 *>(sums) +
                                      (size_t)((i << plan.kshift) * 2 * NB + hb) * 32 + lane;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int u = 0; u < nks; ++u) {
                        const float4 p = r[(size_t)u * 64 * NB];
                        v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
                    }
                    const int s = hb / NB * 8 + g, nrn = up_neuron(item_first(item), s);
                    const int8_t *map = tab.map + item_expert(item) * MOE_MX4_FEW_TOKENS + hb % NB * 8 + 2 * c;
                    if (s < 4 * item_quads(item) && nrn < m) {
                        // approximate division (2 ulp, 0 once 1 + e^-g > 2^126, silu's limit).
                        // h is bf16 as moe_forward's h is, a buffer that callers read: half the
                        // bytes through L2, and y off by 2.4e-3 (rms, of its 64-bit value)
                        // where its own rounding alone makes 1.7e-3
                        if (map[0] >= 0)
                            a.h[(int64_t)map[0] * m8 + nrn] =
                                __float2bfloat16_rn(__fdividef(v.x, 1.0f + __expf(-v.x)) * v.z);
                        if (map[1] >= 0)
                            a.h[(int64_t)map[1] * m8 + nrn] =
                                __float2bfloat16_rn(__fdividef(v.y, 1.0f + __expf(-v.y)) * v.w);
                    }
                }
                if (b1 < plan.n)
                    __syncthreads();  // the sums are read before the next batch's are written
            }
        }
    }

    // ---- h of every CTA complete: a grid barrier; GEMM 2's first weights travel meanwhile,
    // and CTA 0 writes the routing, the tables and the statistics
    __syncthreads();  // h of this CTA is written
    if (threadIdx.x == kThreads - 1)  // releases this CTA's h, ordered before by the barrier above
        asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(a.gbar) : "memory");
    const DownPlan down(a, nsel);
    DownWalk ld(down);
    if (ld.on(down)) {
        down_fill(a, down, ld.strip, tab.sel[ld.is], ld.u * kSlice, ring_s, place);
        ld.next(down);
    }
    if (threadIdx.x == kThreads - 1) {
        uint64_t t0 = 0;
        for (uint32_t i = 1; ld_acquire_u64(a.gbar) < target; ++i) {
            if ((i & 3u) != 0)
                continue;
            const uint64_t now = globaltimer_ns();
            t0 = t0 == 0 ? now : t0;
            if (now - t0 > a.wait_ns) {
                set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                tab.abort = 1;
                break;
            }
        }
    } else if (blockIdx.x == 0 && threadIdx.x < kThreads - 32) {
        constexpr int nt = kThreads - 32;
        const int t1 = (int)threadIdx.x;
        if (t1 < T * k) {
            a.idx[t1] = tab.idx[t1];
            a.w[t1] = tab.w[t1];
            a.slot_row[t1] = tab.slot[t1];
        }
        if (t1 < R)
            a.row_token[t1] = tab.rtok[t1];
        if (t1 <= E)
            a.offsets[t1] = tab.off[t1];
        // the gate statistics, in gate_stats_kernel's arithmetic
        if (t1 < E) {
            float sp = 0.f, sg = 0.f;
            for (int t = 0; t < T; ++t) {
                sp += tab.prob[t * E + t1];
                sg += tab.gw[t * E + t1];
            }
            const int cnt = __popc(tab.mask[t1]);
            a.counts[t1] = cnt;
            a.kept[t1] = tab.off[t1 + 1] - tab.off[t1];
            a.probs_sum[t1] = sp;
            a.importance[t1] = sg;
            a.f[t1] = (float)((double)cnt / ((double)T * k));
            a.P[t1] = (float)((double)sp / (double)T);
        }
        if (t1 == nt - 1) {
            double sfp = 0.0;
            for (int e = 0; e < E; ++e) {
                float sp = 0.f;
                for (int t = 0; t < T; ++t)
                    sp += tab.prob[t * E + e];
                sfp += ((double)__popc(tab.mask[e]) / ((double)T * k)) * ((double)sp / (double)T);
            }
            a.loss[0] = (float)(a.lambda * sfp);
        }
    }
    __syncthreads();

    // ---- GEMM 2 and the combine of this CTA's columns
    if (!tab.abort) {
        uint32_t st = 0;
#pragma unroll 1
        for (int strip = 0; strip < down.strips; ++strip) {
            float acc[2][NB][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[h][nb][q] = 0.f;
            int is = 0, u = warp;
#pragma unroll 1
            while (true) {
                while (u >= down.units) {
                    u -= down.units;
                    ++is;
                }
                if (is >= nsel)
                    break;
                // column t of B: token t's row of this expert, zeros if it has none
                const int8_t *map = tab.map + tab.sel[is] * MOE_MX4_FEW_TOKENS;
                const bf16 *src[NB];
                float w[NB], f[NB][2][2];
                bool on[NB][2];
                uint4 x[NB][8];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const int row = map[nb * 8 + g];
                    src[nb] = row >= 0 ? a.h + (int64_t)row * m8 : nullptr;
                    w[nb] = row >= 0 ? tab.rw[row] : 0.f;
                    // 0 * sum would not do: a NaN weight stays with its tokens
                    on[nb][0] = map[nb * 8 + 2 * c] >= 0;
                    on[nb][1] = map[nb * 8 + 2 * c + 1] >= 0;
                }
                load_b<NB, true>(src, u * kSlice, m, x);
                __syncwarp();  // the other stage has been read
                if (ld.on(down)) {
                    down_fill(a, down, ld.strip, tab.sel[ld.is], ld.u * kSlice, ring_s + (st ^ kStageBytes),
                              place);
                    ld.next(down);
                } else {
                    cp_commit();
                }
                scale_b<NB>(x, u * kSlice, m, w, f);
                cp_wait<1>();
                __syncwarp();
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float sum[NB][4];
                        chunk_mma<NB>(sum, ring_s + st + (2 * h + v) * kChunkBytes, a_off,
                                      [&](int nb, int b) { return x[nb][4 * v + b]; }, g);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (on[nb][j]) {
                                    acc[h][nb][j] = fmaf(sum[nb][j], f[nb][v][j], acc[h][nb][j]);
                                    acc[h][nb][2 + j] = fmaf(sum[nb][2 + j], f[nb][v][j], acc[h][nb][2 + j]);
                                }
                    }
                st ^= kStageBytes;
                u += kWarps;
            }
            if (strip > 0)
                __syncthreads();  // the last strip's sums have been read
            // the warps' sums: [warp][half][nb][lane] float4
            float4 *o = reinterpret_cast<float4 *>(region) + (size_t)warp * 2 * NB * 32 + lane;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    o[(h * NB + nb) * 32] =
                        make_float4(acc[h][nb][0], acc[h][nb][1], acc[h][nb][2], acc[h][nb][3]);
            __syncthreads();
            const float *sums = reinterpret_cast<const float *>(region);
#pragma unroll 1
            for (int j = threadIdx.x; j < 256 * NB; j += kThreads) {
                // j: [half][nb][row bit 3][lane of the fragment][token bit 0]
                const int L = j >> 1 & 31, hn = j >> 7, s = (hn / NB) * 16 + (j >> 6 & 1) * 8 + (L >> 2);
                const int t = hn % NB * 8 + 2 * (L & 3) + (j & 1);
                const int q = down.lo + 8 * strip, col = down_column(q, s);
                if (t < T && s < 4 * (down.hi - q) && col < d) {
                    const float *r = sums + ((size_t)hn * 32 + L) * 4 + (j >> 6 & 1) * 2 + (j & 1);
                    float v = 0.f;
#pragma unroll
                    for (int u = 0; u < kWarps; ++u)
                        v += r[(size_t)u * 2 * NB * 128];
                    a.y[(int64_t)t * d + col] = __float2bfloat16_rn(v * a.scale);
                }
            }
        }
    }
    cp_wait<0>();
}

// --------------------------------------------------------------------- host side

static cudaError_t grid_size(int *out)
{
    static std::mutex mu;
    static int sms[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (sms[dev] == 0) {
        int n = 0;
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(mx4_few_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSmem)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(mx4_few_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSmem)) != cudaSuccess)
            return e;
        sms[dev] = n;
    }
    *out = sms[dev];
    return cudaSuccess;
}

}  // namespace few

bool mx4_few_fits(const moe_params_t *p, bool noisy)
{
    return p->T >= 1 && p->T <= MOE_MX4_FEW_TOKENS && (noisy ? 2 : 1) * p->E <= few::kMaxE;
}

cudaError_t launch_mx4_few(const moe_params_t *p, const moe_mx4_buffers_t *b, char *ws,
                           cudaStream_t s)
{
    using namespace few;
    int grid = 0;
    cudaError_t e = grid_size(&grid);
    if (e != cudaSuccess)
        return e;
    Args a = {};
    a.x = (const bf16 *)b->x;
    a.Wg = (const bf16 *)b->Wg;
    a.Wn = (const bf16 *)b->Wnoise;
    a.noise = b->noise;
    a.bias = b->bias;
    a.W13q = (const uint8_t *)b->W13_q;
    a.W13s = (const uint8_t *)b->W13_s;
    a.W2q = (const uint8_t *)b->W2_q;
    a.W2s = (const uint8_t *)b->W2_s;
    a.h = (bf16 *)b->h;
    a.y = (bf16 *)b->y;
    a.loss = b->loss;
    a.importance = b->importance;
    a.f = b->f;
    a.P = b->P;
    a.probs_sum = b->probs_sum;
    a.w = b->topk_w;
    a.counts = b->counts;
    a.idx = b->topk_idx;
    a.row_token = b->row_token;
    a.slot_row = b->slot_row;
    a.kept = b->kept;
    a.offsets = b->offsets;
    a.status = reinterpret_cast<int32_t *>(ws);
    a.gbar = reinterpret_cast<unsigned long long *>(ws + kWsMx4BarrierWord * 4);
    a.wait_ns = wait_limit_ns();
    a.lambda = p->balance_lambda;
    a.scale = p->rescale ? (float)p->E / (float)p->k : 1.0f;
    a.T = p->T;
    a.d = p->d;
    a.m = p->m;
    a.E = p->E;
    a.k = p->k;
    a.C = p->capacity;
    a.router_type = p->router_type;
    const int64_t r13 = 2 * round_up(p->m, 16);
    a.tk1 = (p->d + 127) / 128;
    a.tk2 = (p->m + 127) / 128;
    a.w13_codes = r13 * (p->d / 2);
    a.w13_scales = (r13 + 127) / 128 * a.tk1 * kMx4Tile;
    a.w2_codes = (int64_t)p->d * (mx4_k32(p->m) / 2);
    a.w2_scales = (int64_t)(p->d + 127) / 128 * a.tk2 * kMx4Tile;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    e = p->T <= 8 ? cudaLaunchKernelEx(&cfg, mx4_few_kernel<1>, a)
                  : cudaLaunchKernelEx(&cfg, mx4_few_kernel<2>, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace moe
