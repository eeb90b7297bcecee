// mx4_few.cu -- the whole layer for 1..16 tokens on mx4 expert weights and bf16
// activations, in one cooperative launch (moe_forward_mx4, MOE_MX4_ACT_BF16).
// Router: "Llama 3 Meets MoE: Efficient Upcycling", section 3 "核心公式" (section 5 for the
// Mixtral and ST types); capacity: its "容量因子"; SwiGLU expert: "LLaMA-MoE v2", code
// sample, class Expert; statistics: "LLaMA-MoE v2", section "门控机制设计".
//
// Bound by the selected experts' weights (0.53 bytes each), then by the chain
// routing -> GEMM 1 -> grid barrier -> GEMM 2.
//
//   routing   every CTA computes all logits (mma.sync on bf16), gates and tables: x and W_g
//             are some ten KB and no CTA waits for another.
//   GEMM 1    the selected experts' neurons are split evenly over the CTAs; an item is 8
//             neurons of one expert: their W1 rows are A rows 0..7 of mma.sync m16n8k16,
//             their W3 rows A rows 8..15, the expert's tokens are B.
//   GEMM 2    after a grid barrier (h complete): each CTA owns a range of output columns of
//             every selected expert (items of 16 W2 rows), so the combine needs no other.
//
// The product.  e2m1 values are exact in f16 (one conversion per pair), so A is the codes
// themselves; B is the bf16 activations scaled by a power of two per row to a maximum in
// [2^13, 2^14): exact in f16 down to 2^-27 of the row's maximum, off by less than 2^-38 of
// it below.  The two products of a 32-column block accumulate in f32 and are added to the
// sum times the block's scale, so the weights' scales may lie any distance apart.  A lane's
// k indexes are 8 consecutive columns, for A and B alike (the order of k inside a product
// is free).
//
// Weights stream through a ring of chunks (16 rows x 128 columns and their 16 scale words)
// that each warp fills for itself with cp.async, several chunks ahead and across items:
// no barrier between loads and products but __syncwarp.  Four warps split the columns of
// an item and four groups of them take the items in turn; partial sums meet in shared
// memory in warp order, so results do not depend on timing.
//
// Rows are enumerated in the order of the scale tiles (4 rows that lie 32 apart share 16
// bytes of scales), so that the scale words of an item fill whole sectors.
#include <mutex>

#include "gate.cuh"
#include "mx4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace few {

using tc::smem_u32;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int KS = 4, NG = kWarps / KS;       // warps that split K, groups of items
constexpr int kChunkCols = 128;
constexpr int kChunkBytes = 16 * 64 + 64;     // codes, scale words
constexpr int kMaxRows = MOE_MX4_FEW_TOKENS * MOE_MAX_TOPK;
constexpr int kMaxE = 32;
constexpr int kMaxDepth = 6;
constexpr int kMinRegion = 32 * 1024;         // the warps' partial logits
constexpr int kMaxRegion = 136 * 1024;
constexpr int kMaxWindow = 4096;              // columns staged at once (a warp's registers)
constexpr size_t kSmemCap = 212 * 1024;       // dynamic; the static tables take 9 KB

struct Args {
    const bf16 *x, *Wg, *Wn;
    const float *noise, *bias;
    const uint8_t *W13q, *W13s, *W2q, *W2s;
    bf16 *h, *y;
    float *loss, *importance, *f, *P, *probs_sum, *w;
    int32_t *counts, *idx, *row_token, *slot_row, *kept, *offsets;
    int32_t *status, *gbar;
    uint64_t wait_ns;
    float lambda, scale;
    int T, d, m, E, k, C, router_type;
    int region, depth, batch, win1, win2;  // bytes; ring chunks; items per reduction; columns
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest depth - 1 groups have landed
__device__ __forceinline__ void cp_wait(int depth)
{
    switch (depth) {
    case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    }
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
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

// pitch (bytes) of staged rows of n columns: 64 mod 128, so that the fragment loads of
// two neighbouring rows fall into different banks
__host__ __device__ inline int row_pitch(int n) { return (2 * n + 127) / 128 * 128 + 64; }

// --------------------------------------------------------------------- work items
// GEMM 1 works on quads of neurons (4 that share 16 bytes of scales), 16 quads per 64
// neurons: quad q is neurons 64 (q / 16) + q % 16 + 16 i.  A CTA takes quads [lo, hi) of
// the selected experts' (expert-major), two per item, items inside one expert.
struct UpItems {
    int lo, hi, per, first;  // per: quads of an expert; first: items in the first expert
    __device__ __forceinline__ UpItems(int nsel, int m)
    {
        per = (m + 63) / 64 * 16;
        const int64_t all = (int64_t)nsel * per;
        lo = (int)(blockIdx.x * all / gridDim.x);
        hi = (int)((blockIdx.x + 1) * all / gridDim.x);
        const int n0 = min(hi - lo, per - (per > 0 ? lo % per : 0));
        first = (n0 + 1) / 2;
    }
    __device__ __forceinline__ int count() const
    {
        const int n0 = min(hi - lo, per - lo % per), rest = hi - lo - n0;
        return first + rest / per * (per / 2) + (rest % per + 1) / 2;
    }
    // item i: its expert (position among the selected), first quad, quads (1 or 2)
    __device__ __forceinline__ void get(int i, int &is, int &q, int &n) const
    {
        int at;  // quad index over all experts
        if (i < first) {
            at = lo + 2 * i;
        } else {
            const int j = i - first;
            at = (lo / per + 1 + j / (per / 2)) * per + 2 * (j % (per / 2));
        }
        is = at / per;
        q = at - is * per;
        n = min(2, min(hi - at, per - q));
    }
};
// neuron s (0..7) of an item that starts at quad q
__device__ __forceinline__ int up_neuron(int q, int s)
{
    const int qq = q + s / 4;
    return qq / 16 * 64 + qq % 16 + 16 * (s % 4);
}

// GEMM 2 works on quads of output columns, 32 quads per 128 columns: quad q is columns
// 128 (q / 32) + q % 32 + 32 i.  A CTA takes quads [lo, hi) of every selected expert, four
// per item.
struct DownItems {
    int lo, hi, per;  // per: items of an expert
    __device__ __forceinline__ explicit DownItems(int d)
    {
        const int64_t all = (d + 127) / 128 * 32;
        lo = (int)(blockIdx.x * all / gridDim.x);
        hi = (int)((blockIdx.x + 1) * all / gridDim.x);
        per = (hi - lo + 3) / 4;
    }
    __device__ __forceinline__ void get(int i, int &is, int &q, int &n) const
    {
        is = i / per;
        q = lo + 4 * (i - is * per);
        n = min(4, hi - q);
    }
};
__device__ __forceinline__ int down_column(int q, int s)
{
    const int qq = q + s / 4;
    return qq / 32 * 128 + qq % 32 + 32 * (s % 4);
}

// --------------------------------------------------------------------- one product phase
// The rows of the weights that A row r (0..15) of item i holds; -1: none.
struct Rows {
    const uint8_t *codes, *scales;  // of the item's expert
    int row;                        // of the expert's matrix, -1 none
};

template <bool UP>
struct Phase {
    const Args &a;
    UpItems up;
    DownItems down;
    int n_items, K32, tk, win, n_win;
    const int32_t *sel;
    __device__ __forceinline__ Phase(const Args &args, int nsel, const int32_t *s_sel)
        : a(args), up(nsel, args.m), down(args.d), sel(s_sel)
    {
        K32 = UP ? a.d : mx4_k32(a.m);
        n_items = nsel == 0 ? 0 : (UP ? (up.hi > up.lo ? up.count() : 0) : nsel * down.per);
        tk = (K32 + 127) / 128;
        win = UP ? a.win1 : a.win2;
        n_win = (K32 + win - 1) / win;
    }
    __device__ __forceinline__ Rows rows(int i, int r) const
    {
        int is, q, n;
        Rows o;
        if constexpr (UP) {
            up.get(i, is, q, n);
            const int e = sel[is], m16 = round_up(a.m, 16), s = r & 7;
            const int nr = up_neuron(q, s);
            o.codes = a.W13q + (int64_t)e * 2 * m16 * (K32 / 2);
            o.scales = a.W13s + (int64_t)e * ((2 * m16 + 127) / 128) * tk * kMx4Tile;
            o.row = (s < 4 * n && nr < a.m) ? (nr / 16) * 32 + nr % 16 + (r >= 8 ? 16 : 0) : -1;
        } else {
            down.get(i, is, q, n);
            const int e = sel[is], col = down_column(q, r);
            o.codes = a.W2q + (int64_t)e * a.d * (K32 / 2);
            o.scales = a.W2s + (int64_t)e * ((a.d + 127) / 128) * tk * kMx4Tile;
            o.row = (r < 4 * n && col < a.d) ? col : -1;
        }
        return o;
    }
    // chunks [lo, hi) of window w that warp ks of a group takes
    __device__ __forceinline__ void share(int w, int ks, int &lo, int &hi) const
    {
        const int c0 = w * (win / kChunkCols);
        const int n = min(win / kChunkCols, tk - c0);
        lo = c0 + ks * n / KS;
        hi = c0 + (ks + 1) * n / KS;
    }
};

// Loader state of one warp: the chunks of a phase in the order the products take them:
// batches of items, windows of columns, the group's items, the warp's chunks.
template <bool UP>
struct Loader {
    const Phase<UP> &p;
    uint32_t ring;       // this warp's stages
    int depth, stage;
    int grp, ks, b0, w, i, c, hi;
    const uint8_t *src0, *src1, *ssrc;  // this lane's 16-byte pieces (two rows), its scale word
    __device__ __forceinline__ Loader(const Phase<UP> &ph, uint32_t r, int dp, int warp)
        : p(ph), ring(r), depth(dp), stage(0), grp(warp / KS), ks(warp % KS), b0(0), w(0), i(grp),
          c(0), hi(0)
    {
        open();
    }
    // moves to the first item and window from (b0, w, i) on that has a chunk
    __device__ __forceinline__ void open()
    {
        while (b0 < p.n_items) {
            int lo;
            p.share(w, ks, lo, hi);
            if (i < min(b0 + p.a.batch, p.n_items) && lo < hi) {
                c = lo;
                const int lane = threadIdx.x & 31;
                const int half = p.K32 / 2;
                const Rows r0 = p.rows(i, lane >> 2), r1 = p.rows(i, (lane >> 2) + 8);
                src0 = r0.row < 0 ? nullptr : r0.codes + (int64_t)r0.row * half + (lane & 3) * 16;
                src1 = r1.row < 0 ? nullptr : r1.codes + (int64_t)r1.row * half + (lane & 3) * 16;
                const Rows rs = p.rows(i, lane & 15);
                ssrc = (lane >= 16 || rs.row < 0)
                           ? nullptr
                           : rs.scales + (int64_t)(rs.row / 128) * p.tk * kMx4Tile +
                                 (rs.row % 32) * 16 + (rs.row % 128) / 32 * 4;
                return;
            }
            if (w + 1 < p.n_win) {
                ++w;
                i = b0 + grp;
            } else {
                b0 += p.a.batch;
                w = 0;
                i = b0 + grp;
            }
        }
    }
    // issues the next chunk (if any) as one group
    __device__ __forceinline__ void issue()
    {
        if (b0 < p.n_items) {
            const int lane = threadIdx.x & 31;
            const uint32_t st = ring + (uint32_t)(stage * kChunkBytes);
            const int row = lane >> 2, piece = lane & 3;
            // columns past K32 are not loaded: their activations are zero
            const bool in = c * 64 + piece * 16 < p.K32 / 2;
            const uint32_t at = (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
            if (in && src0 != nullptr)
                cp16(st + at, src0 + c * 64);
            if (in && src1 != nullptr)
                cp16(st + at + 512, src1 + c * 64);
            if (ssrc != nullptr)
                cp4(st + 1024 + lane * 4, ssrc + (int64_t)c * kMx4Tile);
            if (++c == hi) {
                i += NG;
                if (i >= min(b0 + p.a.batch, p.n_items)) {
                    if (w + 1 < p.n_win) {
                        ++w;
                    } else {
                        b0 += p.a.batch;
                        w = 0;
                    }
                    i = b0 + grp;
                }
                open();
            }
        }
        cp_commit();
        stage = stage + 1 == depth ? 0 : stage + 1;
    }
};

// Stages rows [0, n) (row j from src(j), bf16, columns [c0, c0 + cols) of which those below
// `valid` exist) as f16 scaled by a power of two, zero up to a whole chunk, and the scales'
// inverses in inv[j].  One warp per row; called by the whole CTA between two barriers.
template <class Src>
__device__ __forceinline__ void stage_rows(char *region, int pitch, float *inv, int n, int c0,
                                           int cols, int valid, Src src)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nv = (cols + kChunkCols - 1) / kChunkCols * kChunkCols / 8;  // vectors of a row
    constexpr int V = kMaxWindow / 8 / 32;
    for (int j = warp; j < n; j += kWarps) {
        const bf16 *s = src(j);
        uint4 v[V];
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const int col = c0 + (lane + 32 * q) * 8;
            v[q] = (lane + 32 * q < nv && col < valid)
                       ? __ldcg(reinterpret_cast<const uint4 *>(s + col))
                       : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const int col = c0 + (lane + 32 * q) * 8;
            if (col < valid && col + 8 > valid) {  // h rows: columns past m hold anything
                uint16_t *e = reinterpret_cast<uint16_t *>(&v[q]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + i >= valid)
                        e[i] = 0;
            }
            const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top = max(top, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^(13 - floor(log2(max))): exponent field 127 + 13 - (E - 127), at most 254
        const uint32_t field = min(267u - (top >> 7), 254u);
        const float mul = __uint_as_float(field << 23);
        if (lane == 0)
            inv[j] = mx4_scale(254u - field);
        char *dst = region + (size_t)j * pitch;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            if (lane + 32 * q >= nv)
                break;
            float fv[8];
            bf16x8_to_f32(v[q], fv);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 hh = __floats2half2_rn(fv[2 * i] * mul, fv[2 * i + 1] * mul);
                o[i] = *reinterpret_cast<const uint32_t *>(&hh);
            }
            st_v4(dst + (lane + 32 * q) * 16, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

// acc += A chunk * B: the chunk's 16 rows (stage at `st`) against the token rows at the
// shared addresses bp[nb] (this lane's B row, its 8 columns of block 0 of the chunk).
template <int NB>
__device__ __forceinline__ void chunk_mma(float (&acc)[NB][4], uint32_t st, const uint32_t (&bp)[NB],
                                          int g, int c)
{
    const uint32_t w0 = lds32(st + 1024 + g * 4), w1 = lds32(st + 1024 + (g + 8) * 4);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t at = st + (uint32_t)(g * 64 + ((b ^ ((g >> 1) & 3)) << 4) + c * 4);
        uint32_t a0[4], a1[4];
        mx4_halves8(lds32(at), a0);
        mx4_halves8(lds32(at + 512), a1);
        const float s0 = mx4_scale((w0 >> (8 * b)) & 255u), s1 = mx4_scale((w1 >> (8 * b)) & 255u);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint4 x = lds128(bp[nb] + b * 64);
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(t, a0[0], a1[0], a0[1], a1[1], x.x, x.y);
            mma_f16(t, a0[2], a1[2], a0[3], a1[3], x.z, x.w);
            acc[nb][0] = fmaf(t[0], s0, acc[nb][0]);
            acc[nb][1] = fmaf(t[1], s0, acc[nb][1]);
            acc[nb][2] = fmaf(t[2], s1, acc[nb][2]);
            acc[nb][3] = fmaf(t[3], s1, acc[nb][3]);
        }
    }
}

// --------------------------------------------------------------------- the router
// Logits lg [T][nout] of all tokens: warp w takes 32-column steps [w S / 16, (w + 1) S / 16),
// staging its rows of [W_g | W_noise] in its own `stage` bytes, as many steps at a time as
// fit; the warps' sums are added in warp order (`part`).
template <int NT>
__device__ void router_logits(const Args &a, char *stage, int stage_bytes, float *part, float *lg)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int E = a.E, T = a.T, d = a.d, nout = a.Wn != nullptr ? 2 * E : E;
    constexpr int NP = NT * 8;
    const int steps = d / 32, s_lo = warp * steps / kWarps, s_hi = (warp + 1) * steps / kWarps;
    const int round = stage_bytes / (32 * NP * 2);
    const uint32_t sb = smem_u32(stage);
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            acc[nt][q] = 0.f;
    for (int s0 = s_lo; s0 < s_hi; s0 += round) {
        const int n = min(round, s_hi - s0);
        __syncwarp();
        if ((E & 7) == 0) {  // rows of whole 16-byte pieces
            const int pr = nout / 8, total = n * 32 * pr;
#pragma unroll 4
            for (int i = lane; i < total; i += 32) {
                const int k = i / pr, o = (i - k * pr) * 8;
                const bf16 *src = o < E ? a.Wg + (int64_t)(s0 * 32 + k) * E + o
                                        : a.Wn + (int64_t)(s0 * 32 + k) * E + o - E;
                st_v4(stage + k * NP * 2 + o * 2, ld_nc(src));
            }
        } else {
            const bf16 zero = __float2bfloat16_rn(0.f);
#pragma unroll 4
            for (int i = lane; i < n * 32 * NP; i += 32) {
                const int k = i / NP, o = i - k * NP;
                const int64_t row = (int64_t)(s0 * 32 + k) * E;
                reinterpret_cast<bf16 *>(stage)[i] =
                    o < E ? a.Wg[row + o] : (o < nout ? a.Wn[row + o - E] : zero);
            }
        }
        __syncwarp();
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const bf16 *xs = a.x + (s0 + s) * 32 + 8 * c;
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint4 x0 = g < T ? ld_nc(xs + (int64_t)g * d) : z;
            const uint4 x1 = g + 8 < T ? ld_nc(xs + (int64_t)(g + 8) * d) : z;
            // B of the two products: columns 8c + {0,1 | 2,3} and 8c + {4,5 | 6,7}
            const int i = lane & 7, kk = s * 32 + 8 * (i >> 1) + (i & 1) + 2 * (lane >> 3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t b[4];
                ldsm_x4_trans(sb + (uint32_t)(kk * NP * 2 + nt * 16), b);
                mma_bf16_16816(acc[nt], x0.x, x1.x, x0.y, x1.y, b[0], b[1]);
                mma_bf16_16816(acc[nt], x0.z, x1.z, x0.w, x1.w, b[2], b[3]);
            }
        }
    }
    float *pw = part + (size_t)warp * T * NP;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int o = nt * 8 + 2 * c;
        if (g < T) {
            pw[g * NP + o] = acc[nt][0];
            pw[g * NP + o + 1] = acc[nt][1];
        }
        if (g + 8 < T) {
            pw[(g + 8) * NP + o] = acc[nt][2];
            pw[(g + 8) * NP + o + 1] = acc[nt][3];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * nout; i += kThreads) {
        const int t = i / nout, o = i - t * nout;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            sum += part[((size_t)w * T + t) * NP + o];
        lg[i] = sum;
    }
    __syncthreads();
}

// --------------------------------------------------------------------- the kernel
template <int NB>
__global__ void __launch_bounds__(kThreads, 1) mx4_few_kernel(const __grid_constant__ Args a)
{
    extern __shared__ __align__(128) char sm[];
    __shared__ int32_t s_off[kMaxE + 1], s_sel[kMaxE], s_cnt[kMaxE], s_kept[kMaxE];
    __shared__ int32_t s_idx[kMaxRows], s_slot[kMaxRows], s_rtok[kMaxRows];
    __shared__ float s_w[kMaxRows], s_inv[kMaxRows];
    __shared__ float s_lg[MOE_MX4_FEW_TOKENS * 32], s_prob[MOE_MX4_FEW_TOKENS * kMaxE],
        s_gw[MOE_MX4_FEW_TOKENS * kMaxE];
    __shared__ float s_psum[kMaxE], s_imp[kMaxE];
    __shared__ int s_nsel, s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int T = a.T, E = a.E, k = a.k, d = a.d, m = a.m;
    constexpr int RQ = 4 * NB;                      // sums of a lane
    char *region = sm;
    float *red = reinterpret_cast<float *>(sm + a.region);
    char *ring = sm + a.region + a.batch * KS * 32 * RQ * 4;
    float *outs = reinterpret_cast<float *>(ring + kWarps * a.depth * kChunkBytes);
    char *my_ring = ring + warp * a.depth * kChunkBytes;
    if (threadIdx.x == 0)
        s_abort = 0;
    // the grid barrier's generation before this launch's barrier (it changes only once
    // every CTA has arrived, this one included)
    int32_t gen = 0;
    if (threadIdx.x == 0)
        gen = ld_acquire_gpu(a.gbar + 1);

    // ---- router
    const int nout = a.Wn != nullptr ? 2 * E : E;
    float *part = reinterpret_cast<float *>(region);
    const int sbytes = a.depth * kChunkBytes;
    switch ((nout + 7) / 8) {
    case 1: router_logits<1>(a, my_ring, sbytes, part, s_lg); break;
    case 2: router_logits<2>(a, my_ring, sbytes, part, s_lg); break;
    case 3: router_logits<3>(a, my_ring, sbytes, part, s_lg); break;
    default: router_logits<4>(a, my_ring, sbytes, part, s_lg); break;
    }
    if (warp < T)
        gate_token_warp(s_lg + warp * nout, E, k, a.Wn != nullptr ? 1 : 0,
                        a.noise + (a.noise != nullptr ? (size_t)warp * E : 0), a.bias, a.router_type,
                        s_idx + warp * k, s_w + warp * k, s_prob + warp * E, s_gw + warp * E,
                        a.status);
    __syncthreads();
    // ---- dispatch tables: stable by token, assignments past the capacity dropped
    if (threadIdx.x < E) {
        const int e = threadIdx.x;
        int cnt = 0;
        float sp = 0.f, sg = 0.f;
        for (int i = 0; i < T * k; ++i)
            cnt += s_idx[i] == e;
        for (int t = 0; t < T; ++t) {
            sp += s_prob[t * E + e];
            sg += s_gw[t * E + e];
        }
        s_cnt[e] = cnt;
        s_kept[e] = a.C < 0 ? cnt : min(cnt, a.C);
        s_psum[e] = sp;
        s_imp[e] = sg;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int acc = 0, ns = 0;
        for (int e = 0; e < E; ++e) {
            s_off[e] = acc;
            acc += s_kept[e];
            if (s_kept[e] > 0)
                s_sel[ns++] = e;
        }
        s_off[E] = acc;
        s_nsel = ns;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += kThreads) {
        const int t = i / k, e = s_idx[i];
        int row = -1;
        if (e >= 0 && e < E) {
            int rank = 0;  // the expert's assignments of earlier tokens
            for (int j = 0; j < t * k; ++j)
                rank += s_idx[j] == e;
            if (rank < s_kept[e]) {
                row = s_off[e] + rank;
                s_rtok[row] = t;
            }
        }
        s_slot[i] = row;
    }
    __syncthreads();
    const int nsel = s_nsel, R = s_off[E], m8 = round_up(m, 8);

    // ---- one product phase: every item's sums, handed to done(item, sum) where
    // sum(L, q) is value q of lane L
    auto products = [&](auto &ph, auto &ld, int pitch, auto stage, auto brow, auto done) {
        const int grp = warp / KS, ks = warp % KS;
        int st = 0;
        bool staged = false;
        for (int b0 = 0; b0 < ph.n_items; b0 += a.batch) {
            const int b1 = min(b0 + a.batch, ph.n_items);
            for (int w = 0; w < ph.n_win; ++w) {
                if (!staged || ph.n_win > 1) {
                    if (staged)
                        __syncthreads();  // the last window's products are done
                    stage(w);
                    __syncthreads();
                    staged = true;
                }
                int lo, hi;
                ph.share(w, ks, lo, hi);
                const int c0 = w * (ph.win / kChunkCols);
                for (int i = b0 + grp; i < b1; i += NG) {
                    uint32_t bp0[NB];
                    int brw[NB][2];
                    brow(i, bp0, brw);
                    float acc[NB][4];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[nb][q] = 0.f;
                    for (int ch = lo; ch < hi; ++ch) {
                        __syncwarp();  // the stage the loader fills next has been read
                        ld.issue();
                        cp_wait(a.depth);
                        __syncwarp();
                        uint32_t bp[NB];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            bp[nb] = bp0[nb] + (uint32_t)((ch - c0) * kChunkCols * 2 + 16 * c);
                        chunk_mma<NB>(acc, smem_u32(my_ring) + (uint32_t)(st * kChunkBytes), bp, g, c);
                        st = st + 1 == a.depth ? 0 : st + 1;
                    }
                    float *rw = red + ((size_t)((i - b0) * KS + ks) * 32 + lane) * RQ;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float v = acc[nb][q] * s_inv[brw[nb][q & 1]];
                            rw[nb * 4 + q] = w == 0 ? v : rw[nb * 4 + q] + v;
                        }
                }
            }
            __syncthreads();
            for (int i = b0; i < b1; ++i)
                done(i, [&](int L, int q) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        s += red[((size_t)((i - b0) * KS + j) * 32 + L) * RQ + q];
                    return s;
                });
            if (b1 < ph.n_items)
                __syncthreads();  // the sums are read before the next batch's are written
        }
    };

    // ---- GEMM 1
    const int pitch1 = row_pitch(a.win1), pitch2 = row_pitch(a.win2);
    const uint32_t region_s = smem_u32(region);
    {
        const Phase<true> ph(a, nsel, s_sel);
        Loader<true> ld(ph, smem_u32(my_ring), a.depth, warp);
        for (int i = 0; i < a.depth - 1; ++i)
            ld.issue();
        products(
            ph, ld, pitch1,
            [&](int w) {
                stage_rows(region, pitch1, s_inv, T, w * a.win1, min(a.win1, d - w * a.win1), d,
                           [&](int j) { return a.x + (int64_t)j * d; });
            },
            [&](int i, uint32_t (&bp)[NB], int (&br)[NB][2]) {
                int is, q, n;
                ph.up.get(i, is, q, n);
                const int e = s_sel[is], r0 = s_off[e], nr = s_off[e + 1] - r0;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    bp[nb] = region_s + (uint32_t)(s_rtok[r0 + min(nb * 8 + g, nr - 1)] * pitch1);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        br[nb][j] = s_rtok[r0 + min(nb * 8 + 2 * c + j, nr - 1)];
                }
            },
            [&](int i, auto sum) {
                int is, q, n;
                ph.up.get(i, is, q, n);
                const int e = s_sel[is], r0 = s_off[e], nr = s_off[e + 1] - r0;
                if (threadIdx.x < 64 * NB) {
                    const int s = threadIdx.x & 7, tok = threadIdx.x >> 3;
                    const int nrn = up_neuron(q, s), L = s * 4 + (tok & 7) / 2, at = tok / 8 * 4 + (tok & 1);
                    if (s < 4 * n && nrn < m && tok < nr) {
                        const float gv = sum(L, at), uv = sum(L, at + 2);
                        // approximate division (2 ulp, 0 once 1 + e^-g > 2^126, silu's limit)
                        a.h[(int64_t)(r0 + tok) * m8 + nrn] =
                            __float2bfloat16_rn(__fdividef(gv, 1.0f + __expf(-gv)) * uv);
                    }
                }
            });
    }

    // ---- h of every CTA complete: a grid barrier; GEMM 2's first weights travel meanwhile,
    // and CTA 0 writes the routing, the tables and the statistics
    const Phase<false> ph(a, nsel, s_sel);
    __syncwarp();
    Loader<false> ld(ph, smem_u32(my_ring), a.depth, warp);
    for (int i = 0; i < a.depth - 1; ++i)
        ld.issue();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int G = (int)gridDim.x;
        __threadfence();  // this CTA's h, ordered before by the barrier above
        if (atomicAdd(a.gbar, 1) == G - 1) {  // the last to arrive releases the others
            __threadfence();
            atomicAdd(a.gbar + 1, 1);
            asm volatile("red.relaxed.gpu.global.and.b32 [%0], 0;" ::"l"(a.gbar) : "memory");
        } else {
            const uint64_t t0 = globaltimer_ns();
            while (ld_acquire_gpu(a.gbar + 1) == gen) {
                if (globaltimer_ns() - t0 > a.wait_ns) {
                    set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    s_abort = 1;
                    break;
                }
                __nanosleep(32);
            }
        }
    } else if (blockIdx.x == 0) {
        const int nt = kThreads - 32, t1 = (int)threadIdx.x - 32;
        if (t1 >= 0) {
            for (int i = t1; i < T * k; i += nt) {
                a.idx[i] = s_idx[i];
                a.w[i] = s_w[i];
                a.slot_row[i] = s_slot[i];
            }
            for (int r = t1; r < R; r += nt)
                a.row_token[r] = s_rtok[r];
            for (int e = t1; e <= E; e += nt)
                a.offsets[e] = s_off[e];
            // the gate statistics, in gate_stats_kernel's arithmetic
            for (int e = t1; e < E; e += nt) {
                a.counts[e] = s_cnt[e];
                a.kept[e] = s_kept[e];
                a.probs_sum[e] = s_psum[e];
                a.importance[e] = s_imp[e];
                a.f[e] = (float)((double)s_cnt[e] / ((double)T * k));
                a.P[e] = (float)((double)s_psum[e] / (double)T);
            }
            if (t1 == nt - 1) {
                double sfp = 0.0;
                for (int e = 0; e < E; ++e)
                    sfp += ((double)s_cnt[e] / ((double)T * k)) * ((double)s_psum[e] / (double)T);
                a.loss[0] = (float)(a.lambda * sfp);
            }
        }
    }
    __syncthreads();

    // ---- GEMM 2 and the combine of this CTA's columns
    if (!s_abort) {
        const int ncol = 4 * (ph.down.hi - ph.down.lo);
        products(
            ph, ld, pitch2,
            [&](int w) {
                const int K = mx4_k32(m);
                stage_rows(region, pitch2, s_inv, R, w * a.win2, min(a.win2, K - w * a.win2), m,
                           [&](int j) { return a.h + (int64_t)j * m8; });
            },
            [&](int i, uint32_t (&bp)[NB], int (&br)[NB][2]) {
                const int e = s_sel[i / ph.down.per], r0 = s_off[e], nr = s_off[e + 1] - r0;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    bp[nb] = region_s + (uint32_t)((r0 + min(nb * 8 + g, nr - 1)) * pitch2);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        br[nb][j] = r0 + min(nb * 8 + 2 * c + j, nr - 1);
                }
            },
            [&](int i, auto sum) {
                int is, q, n;
                ph.down.get(i, is, q, n);
                const int e = s_sel[is], r0 = s_off[e], nr = s_off[e + 1] - r0;
                if (threadIdx.x < 128 * NB) {
                    const int s = threadIdx.x & 15, tok = threadIdx.x >> 4;
                    const int L = (s & 7) * 4 + (tok & 7) / 2, at = tok / 8 * 4 + (tok & 1) + (s & 8) / 4;
                    if (s < 4 * n && tok < nr)
                        outs[(size_t)(r0 + tok) * ncol + 4 * (q - ph.down.lo) + s] = sum(L, at);
                }
            });
        __syncthreads();
        for (int i = threadIdx.x; i < T * ncol; i += kThreads) {
            const int t = i / ncol, o = i - t * ncol;
            const int col = down_column(ph.down.lo, o);
            if (col >= d)
                continue;
            float acc = 0.f;
            for (int j = 0; j < k; ++j) {
                const int row = s_slot[t * k + j];
                if (row >= 0)
                    acc = fmaf(s_w[t * k + j], outs[(size_t)row * ncol + o], acc);
            }
            a.y[(int64_t)t * d + col] = __float2bfloat16_rn(acc * a.scale);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
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
                                      (int)kSmemCap)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(mx4_few_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)kSmemCap)) != cudaSuccess)
            return e;
        sms[dev] = n;
    }
    *out = sms[dev];
    return cudaSuccess;
}

// Columns staged at once for `rows` activation rows of K columns: all of them if they fit
// the region and a warp's registers, else as many whole chunks as do.
static int window(int rows, int K)
{
    const int k128 = (K + kChunkCols - 1) / kChunkCols * kChunkCols;
    int w = (kMaxRegion / rows - 64) / 2 / kChunkCols * kChunkCols;
    w = w < kMaxWindow ? w : kMaxWindow;
    return w < k128 ? w : k128;
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
    a.gbar = a.status + kWsDecodeBarrierWord;
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
    const int R = p->T * p->k, nb = p->T <= 8 ? 1 : 2;
    a.win1 = window(p->T, p->d);
    a.win2 = window(R, p->m);
    const int x_bytes = p->T * row_pitch(a.win1), h_bytes = R * row_pitch(a.win2);
    a.region = round_up(x_bytes > h_bytes ? x_bytes : h_bytes, 128);
    a.region = a.region > kMinRegion ? a.region : kMinRegion;
    a.batch = nb == 1 ? 8 : 4;
    const size_t red = (size_t)a.batch * KS * 32 * 4 * nb * 4;
    const int64_t quads = (p->d + 127) / 128 * 32;
    const size_t outs = (size_t)R * 4 * ((quads + grid - 1) / grid + 1) * 4;
    const size_t fixed = a.region + red + outs;
    const size_t per = (size_t)kWarps * kChunkBytes;
    if (fixed + 2 * per > kSmemCap)
        return cudaErrorInvalidValue;
    a.depth = (int)((kSmemCap - fixed) / per);
    a.depth = a.depth < kMaxDepth ? a.depth : kMaxDepth;
    const size_t smem = fixed + a.depth * per;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    e = nb == 1 ? cudaLaunchKernelEx(&cfg, mx4_few_kernel<1>, a)
                : cudaLaunchKernelEx(&cfg, mx4_few_kernel<2>, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace moe
