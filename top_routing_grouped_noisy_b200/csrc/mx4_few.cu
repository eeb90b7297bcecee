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
#include <type_traits>

#include "gate.cuh"
#include "mx4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace few {

using tc::smem_u32;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kChunkCols = 128;
constexpr int kChunkBytes = 16 * 64 + 64;     // codes, scale words
// chunks of a ring stage: two halve the loop's overhead per weight; with two groups of 8
// tokens the staged activations leave room for single chunks only
__host__ __device__ constexpr int stage_chunks(int nb) { return nb == 1 ? 2 : 1; }
__host__ __device__ constexpr int stage_cols(int nb) { return stage_chunks(nb) * kChunkCols; }
__host__ __device__ constexpr int stage_bytes(int nb) { return stage_chunks(nb) * kChunkBytes; }
constexpr int kMaxRows = MOE_MX4_FEW_TOKENS * MOE_MAX_TOPK;
constexpr int kMaxE = 32;
constexpr int kMaxRegion = 136 * 1024;        // staged activations
constexpr int kMaxWindow = 8192;              // columns staged at once
constexpr int kMaxInv = 1088;                 // (row, chunk) scales of a window
constexpr size_t kSmemCap = 212 * 1024;       // dynamic; the static tables take 12 KB

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
    int region, red, win1, win2;  // bytes, bytes, columns staged
};

// 16 or 4 bytes to shared memory; zeros where `on` is false (nothing is read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 4 : 0)
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
        const uint32_t all = (uint32_t)(nsel * per);  // at most 2^23, times the grid below 2^32
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
        const uint32_t all = (uint32_t)((d + 127) / 128 * 32);
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
// Items of a phase, at most kItems at a time, as a table in shared memory: expert, quads and
// first quad packed into a word (the divisions behind them are made once per item, not by
// every lane that loads or multiplies it).
constexpr int kItems = 512;
__device__ __forceinline__ int32_t item_pack(int e, int q, int n) { return e | n << 5 | q << 8; }
__device__ __forceinline__ int item_expert(int32_t v) { return v & 31; }
__device__ __forceinline__ int item_quads(int32_t v) { return v >> 5 & 7; }
__device__ __forceinline__ int item_first(int32_t v) { return v >> 8; }

template <bool UP, int NB>
struct Phase {
    const Args &a;
    const int32_t *items;
    int n_items;                    // in the table
    int kshift;                     // 2^kshift warps (a group) split the columns of an item
    int K32, tk, win, n_win;
    const uint8_t *codes, *scales;  // of all experts
    int64_t codes_e, scales_e;      // bytes of an expert's
    __device__ __forceinline__ Phase(const Args &args, const int32_t *table)
        : a(args), items(table), n_items(0), kshift(0)
    {
        const int rows = UP ? 2 * round_up(a.m, 16) : a.d;
        K32 = UP ? a.d : mx4_k32(a.m);
        tk = (K32 + 127) / 128;
        win = UP ? a.win1 : a.win2;
        n_win = (K32 + win - 1) / win;
        codes = UP ? a.W13q : a.W2q;
        scales = UP ? a.W13s : a.W2s;
        codes_e = (int64_t)rows * (K32 / 2);
        scales_e = (int64_t)((rows + 127) / 128) * tk * kMx4Tile;
    }
    // For n items in the table: the split with the fewest stages on the busiest warp (the
    // items go round the 16 / 2^kshift groups), the sum of an item's parts counted as half a
    // stage.
    __device__ __forceinline__ void set(int n)
    {
        n_items = n;
        const int steps = n_win * ((min(win, K32) + stage_cols(NB) - 1) / stage_cols(NB));
        int best = 1 << 30;
#pragma unroll
        for (int k = 0; k <= 4; ++k) {
            const int cost = ((n + (kWarps >> k) - 1) >> (4 - k)) *
                             (2 * ((steps + (1 << k) - 1) >> k) + (k > 0 ? 1 : 0));
            if (cost < best) {
                best = cost;
                kshift = k;
            }
        }
    }
    // the row of the expert's matrix that A row r (0..15) of an item holds; -1: none
    __device__ __forceinline__ int row(int32_t item, int r) const
    {
        const int q = item_first(item), n4 = 4 * item_quads(item);
        if constexpr (UP) {
            const int s = r & 7, nr = up_neuron(q, s);
            return (s < n4 && nr < a.m) ? (nr >> 4) * 32 + (nr & 15) + (r >= 8 ? 16 : 0) : -1;
        } else {
            const int col = down_column(q, r);
            return (r < n4 && col < a.d) ? col : -1;
        }
    }
    // stages [lo, hi) of window w (counted inside it) that this warp takes
    __device__ __forceinline__ void share(int w, int &lo, int &hi) const
    {
        const int n = (min(win, K32 - w * win) + stage_cols(NB) - 1) / stage_cols(NB);
        const int ks = (int)(threadIdx.x >> 5) & ((1 << kshift) - 1);
        lo = (ks * n) >> kshift;
        hi = ((ks + 1) * n) >> kshift;
    }
    // chunks staged of window w: whole stages
    __device__ __forceinline__ int chunks(int w) const
    {
        return (min(win, K32 - w * win) + stage_cols(NB) - 1) / stage_cols(NB) * stage_chunks(NB);
    }
    __device__ __forceinline__ int group() const { return (int)(threadIdx.x >> 5) >> kshift; }
    __device__ __forceinline__ int groups() const { return kWarps >> kshift; }
};

// Loader state of one warp: the stages of a phase's table in the order the products take
// them: the group's items, windows of columns, the warp's stages.
template <bool UP, int NB, int DEPTH>
struct Loader {
    static constexpr int SB = stage_bytes(NB), SC = stage_chunks(NB);
    const Phase<UP, NB> &p;
    uint32_t ring, st, dst;  // this warp's stages, the next one, this lane's place in it
    int w, i, c, hi;         // c: first chunk of the next stage; hi: end of the warp's share
    const uint8_t *src0, *src1, *ssrc;  // this lane's 16-byte pieces (two rows), its scale word
    bool on0, on1, ons;
    __device__ __forceinline__ Loader(const Phase<UP, NB> &ph, uint32_t r)
        : p(ph), ring(r), w(0)
    {
        const int lane = threadIdx.x & 31, row = lane >> 2, piece = lane & 3;
        dst = (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
        restart();
    }
    // from the start of a (refilled) table: the first stages of the ring
    __device__ __forceinline__ void restart()
    {
        w = 0;
        st = ring;
        i = p.group();
        open();
#pragma unroll 1
        for (int n = 0; n < DEPTH - 1; ++n)
            issue();
    }
    // moves to the first item and window from (i, w) on that has a stage
    __device__ __forceinline__ void open()
    {
        while (i < p.n_items) {
            int lo;
            p.share(w, lo, hi);
            if (lo < hi) {
                const int cw = w * (p.win / kChunkCols);
                c = cw + lo * SC;
                hi = cw + hi * SC;
                const int lane = threadIdx.x & 31;
                const int32_t item = p.items[i];
                const int e = item_expert(item);
                const int r0 = p.row(item, lane >> 2), r1 = p.row(item, (lane >> 2) + 8);
                const int rs = p.row(item, lane & 15);
                on0 = r0 >= 0;
                on1 = r1 >= 0;
                ons = rs >= 0;
                const uint8_t *ce = p.codes + e * p.codes_e + (lane & 3) * 16 + c * 64;
                src0 = ce + (int64_t)max(r0, 0) * (p.K32 / 2);
                src1 = ce + (int64_t)max(r1, 0) * (p.K32 / 2);
                const int q = max(rs, 0);
                // lanes 0..15: the words of the stage's first chunk; 16..31: of its second
                ssrc = p.scales + e * p.scales_e +
                       ((int64_t)(q >> 7) * p.tk + c + (lane >> 4)) * kMx4Tile + (q & 31) * 16 +
                       (q >> 5 & 3) * 4;
                return;
            }
            next();
        }
    }
    __device__ __forceinline__ void next()
    {
        if (++w == p.n_win) {
            w = 0;
            i += p.groups();
        }
    }
    // issues the next stage (if any) as one group
    __device__ __forceinline__ void issue()
    {
        if (i < p.n_items) {
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int u = 0; u < SC; ++u) {  // columns past K32 are zeros
                const bool in = (c + u) * 64 + (lane & 3) * 16 < p.K32 / 2;
                cp16(st + u * kChunkBytes + dst, src0 + u * 64, in && on0);
                cp16(st + u * kChunkBytes + dst + 512, src1 + u * 64, in && on1);
            }
            if (SC == 2 || lane < 16)
                cp4(st + (lane >> 4) * kChunkBytes + 1024 + (lane & 15) * 4, ssrc,
                    ons && c + (lane >> 4) < p.tk);
            src0 += SC * 64;
            src1 += SC * 64;
            ssrc += SC * kMx4Tile;
            c += SC;
            if (__builtin_expect(c == hi, 0)) {
                next();
                open();
            }
        }
        cp_commit();
        st = st + SB == ring + DEPTH * SB ? ring : st + SB;
    }
};

// One chunk (128 columns) of one staged row, 16 lanes with 8 bf16 columns each, as f16 scaled
// by a power of two to a maximum in [2^13, 2^14); returns the scale's inverse.
__device__ __forceinline__ float scale_chunk(uint4 &v)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = max(top, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 2^(13 - floor(log2(max))): exponent field 127 + 13 - (E - 127), at most 254
    const uint32_t field = min(267u - (top >> 7), 254u);
    const float mul = __uint_as_float(field << 23);
    float f[8];
    bf16x8_to_f32(v, f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 hh = __floats2half2_rn(f[2 * i] * mul, f[2 * i + 1] * mul);
        o[i] = *reinterpret_cast<const uint32_t *>(&hh);
    }
    v = make_uint4(o[0], o[1], o[2], o[3]);
    return mx4_scale(254u - field);
}

// Stages rows [0, n), `chunks` chunks from column c0 (row j at src + j ld, columns below
// `valid` exist, zeros past them) as scaled f16, inv[j * chunks + ch] the scales' inverses.  With RAW the bf16 rows lie in the region already.  Called by warps
// [first, 16), each half warp one chunk of one row at a time.
template <bool RAW>
__device__ __forceinline__ void stage_rows(char *region, int pitch, float *inv, int n, int c0,
                                           int chunks, int valid, const bf16 *src, int64_t ld,
                                           int first)
{
    const int total = n * chunks;
    const int hw = ((int)threadIdx.x >> 4) - 2 * first, l = threadIdx.x & 15;
    const int step = 2 * (kWarps - first);
    constexpr int U = 4;
#pragma unroll 1
    for (int i0 = hw & ~1; i0 < total; i0 += U * step) {  // both halves of a warp loop alike
        uint4 v[U];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + (hw & 1) + u * step;
            const int j = i / chunks, col = (i - j * chunks) * kChunkCols + 8 * l;
            at[u] = i < total ? j * pitch + col * 2 : -1;
            v[u] = make_uint4(0, 0, 0, 0);
            if (i < total && c0 + col < valid)
                v[u] = RAW ? *reinterpret_cast<const uint4 *>(region + at[u])
                           : __ldcg(reinterpret_cast<const uint4 *>(src + j * ld + c0 + col));
            if (!RAW && c0 + col + 8 > valid) {  // columns past the row's end hold anything
                uint16_t *e = reinterpret_cast<uint16_t *>(&v[u]);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (c0 + col + q >= valid)
                        e[q] = 0;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float r = scale_chunk(v[u]);
            if (at[u] >= 0) {
                st_v4(region + at[u], v[u]);
                if (l == 0)
                    inv[i0 + (hw & 1) + u * step] = r;
            }
        }
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

// acc += (A chunk * B) * inv: the chunk's 16 rows (stage at `st`, this lane's words of row g
// at off[b]) against the token rows at the shared addresses bp[nb] (this lane's B row and 8
// columns); inv[nb][j]: the scale of the row of token 2c + j.
template <int NB>
__device__ __forceinline__ void chunk_mma(float (&acc)[NB][4], uint32_t st, const uint32_t (&off)[4],
                                          const uint32_t (&bp)[NB], const uint32_t (&ip)[NB][2],
                                          int g)
{
    float s0[4], s1[4];
    word_scales(lds32(st + 1024 + g * 4), s0);
    word_scales(lds32(st + 1056 + g * 4), s1);
    float sum[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sum[nb][q] = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        uint32_t a0[4], a1[4];
        mx4_halves8(lds32(st + off[b]), a0);
        mx4_halves8(lds32(st + off[b] + 512), a1);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const uint4 x = lds128(bp[nb] + b * 64);
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(t, a0[0], a1[0], a0[1], a1[1], x.x, x.y);
            mma_f16(t, a0[2], a1[2], a0[3], a1[3], x.z, x.w);
            sum[nb][0] = fmaf(t[0], s0[b], sum[nb][0]);
            sum[nb][1] = fmaf(t[1], s0[b], sum[nb][1]);
            sum[nb][2] = fmaf(t[2], s1[b], sum[nb][2]);
            sum[nb][3] = fmaf(t[3], s1[b], sum[nb][3]);
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float i0 = __uint_as_float(lds32(ip[nb][0])), i1 = __uint_as_float(lds32(ip[nb][1]));
        acc[nb][0] = fmaf(sum[nb][0], i0, acc[nb][0]);
        acc[nb][1] = fmaf(sum[nb][1], i1, acc[nb][1]);
        acc[nb][2] = fmaf(sum[nb][2], i0, acc[nb][2]);
        acc[nb][3] = fmaf(sum[nb][3], i1, acc[nb][3]);
    }
}

// --------------------------------------------------------------------- the router
// Adds the 32-column steps [s_lo, s_hi) of a window whose bf16 rows lie in the region (step
// 0 at its start, at global column c0) into acc: the warp's rows of [W_g | W_noise] go to its
// own `stage` bytes, as many steps at a time as fit.
template <int NT>
__device__ __forceinline__ void router_steps(const Args &a, uint32_t rows, int pitch, int c0,
                                             int s_lo, int s_hi, char *stage, int stage_bytes,
                                             float (&acc)[NT][4])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int E = a.E, T = a.T, nout = a.Wn != nullptr ? 2 * E : E;
    constexpr int NP = NT * 8;
    const int round = stage_bytes / (32 * NP * 2);
    const uint32_t sb = smem_u32(stage);
#pragma unroll 1
    for (int s0 = s_lo; s0 < s_hi; s0 += round) {
        const int n = min(round, s_hi - s0);
        const int64_t k0 = c0 + s0 * 32;
        __syncwarp();
        if ((E & 7) == 0) {  // rows of whole 16-byte pieces
            constexpr int PR = NT;
#pragma unroll 4
            for (int i = lane; i < n * 32 * PR; i += 32) {
                const int k = i / PR, o = (i % PR) * 8;
                const bf16 *src = o < E ? a.Wg + (k0 + k) * E + o : a.Wn + (k0 + k) * E + o - E;
                cp16(sb + i * 16, src, true);
            }
            cp_commit();
            cp_wait<0>();
        } else {
            const bf16 zero = __float2bfloat16_rn(0.f);
#pragma unroll 4
            for (int i = lane; i < n * 32 * NP; i += 32) {
                const int k = i / NP, o = i % NP;
                reinterpret_cast<bf16 *>(stage)[i] =
                    o < E ? a.Wg[(k0 + k) * E + o]
                          : (o < nout ? a.Wn[(k0 + k) * E + o - E] : zero);
            }
        }
        __syncwarp();
#pragma unroll 2
        for (int s = 0; s < n; ++s) {
            // A: 8 consecutive columns of token rows g, g + 8; B of the two products:
            // columns 8c + {0,1 | 2,3} and 8c + {4,5 | 6,7}
            const uint32_t xa = rows + (uint32_t)(g * pitch + ((s0 + s) * 32 + 8 * c) * 2);
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint4 x0 = g < T ? lds128(xa) : z;
            const uint4 x1 = g + 8 < T ? lds128(xa + 8 * pitch) : z;
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
}

// Copies columns [c0, c0 + cols) of x's rows into the region as they are (asynchronous, one
// group per thread).
__device__ __forceinline__ void load_x(const Args &a, uint32_t region, int pitch, int c0, int cols)
{
    const int nv = cols / 8;
#pragma unroll 1
    for (int t = 0; t < a.T; ++t)
#pragma unroll 2
        for (int v = threadIdx.x; v < nv; v += kThreads)
            cp16(region + (uint32_t)(t * pitch + v * 16), a.x + (int64_t)t * a.d + c0 + v * 8, true);
    cp_commit();
}

// The logits lg [T][nout] of all tokens: in every window of x, warp w takes the w-th
// sixteenth of the 32-column steps; the warps' sums are added in warp order.  With one window
// the region is left holding x.
template <int NT>
__device__ __noinline__ void router_logits(const Args &a, char *region, int pitch, char *stage,
                                           int stage_bytes, float *part, float *lg)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int T = a.T, nout = a.Wn != nullptr ? 2 * a.E : a.E;
    constexpr int NP = NT * 8;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            acc[nt][q] = 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < a.d; c0 += a.win1) {
        const int cols = min(a.win1, a.d - c0), steps = cols / 32;
        if (c0 > 0) {
            __syncthreads();  // the last window's rows have been read
            load_x(a, smem_u32(region), pitch, c0, cols);
        }
        cp_wait<0>();
        __syncthreads();
        router_steps<NT>(a, smem_u32(region), pitch, c0, warp * steps / kWarps,
                         (warp + 1) * steps / kWarps, stage, stage_bytes, acc);
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
template <int NB, int DEPTH>
__global__ void __launch_bounds__(kThreads, 1) mx4_few_kernel(const __grid_constant__ Args a)
{
    extern __shared__ __align__(128) char sm[];
    __shared__ int32_t s_off[kMaxE + 1], s_sel[kMaxE], s_cnt[kMaxE], s_kept[kMaxE];
    __shared__ int32_t s_idx[kMaxRows], s_slot[kMaxRows], s_rtok[kMaxRows];
    __shared__ float s_w[kMaxRows], s_inv[kMaxInv];
    __shared__ float s_lg[MOE_MX4_FEW_TOKENS * 32], s_prob[MOE_MX4_FEW_TOKENS * kMaxE],
        s_gw[MOE_MX4_FEW_TOKENS * kMaxE];
    __shared__ int32_t s_items[kItems];
    __shared__ int s_nsel, s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int T = a.T, E = a.E, k = a.k, d = a.d, m = a.m;
    constexpr int RQ = 4 * NB;                      // sums of a lane
    char *region = sm;
    float *red = reinterpret_cast<float *>(sm + a.region);
    constexpr int SB = stage_bytes(NB), SC = stage_chunks(NB);
    char *ring = sm + a.region + a.red;
    float *outs = reinterpret_cast<float *>(ring + kWarps * DEPTH * SB);
    char *my_ring = ring + warp * DEPTH * SB;
    const int pitch1 = row_pitch(a.win1), pitch2 = row_pitch(a.win2);
    const uint32_t region_s = smem_u32(region), ring_s = smem_u32(my_ring);
    load_x(a, region_s, pitch1, 0, min(a.win1, d));
    // the grid barrier's generation before this launch's barrier (it changes only once
    // every CTA has arrived, this one included)
    int32_t gen = 0;
    if (threadIdx.x == 0) {
        s_abort = 0;
        gen = ld_acquire_gpu(a.gbar + 1);
    }

    // ---- router
    const int nout = a.Wn != nullptr ? 2 * E : E;
    switch ((nout + 7) / 8) {
    case 1: router_logits<1>(a, region, pitch1, my_ring, DEPTH * SB, red, s_lg); break;
    case 2: router_logits<2>(a, region, pitch1, my_ring, DEPTH * SB, red, s_lg); break;
    case 3: router_logits<3>(a, region, pitch1, my_ring, DEPTH * SB, red, s_lg); break;
    default: router_logits<4>(a, region, pitch1, my_ring, DEPTH * SB, red, s_lg); break;
    }
    if (warp < T)
        gate_token_warp(s_lg + warp * nout, E, k, a.Wn != nullptr ? 1 : 0,
                        a.noise + (a.noise != nullptr ? (size_t)warp * E : 0), a.bias, a.router_type,
                        s_idx + warp * k, s_w + warp * k, s_prob + warp * E, s_gw + warp * E,
                        a.status);
    __syncthreads();
    // ---- dispatch tables by warp 0 (lane e: expert e): stable by token, assignments past the
    // capacity dropped; the other warps turn the staged x into scaled f16
    const bool one_window = d <= a.win1;
    const int chunks1 = (min(a.win1, d) + stage_cols(NB) - 1) / stage_cols(NB) * SC;
    if (warp == 0) {
        constexpr int B = kMaxRows / 32;
        const int n = T * k;
        int v[B], rank[B], cnt = 0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            v[b] = 32 * b + lane < n ? s_idx[32 * b + lane] : -1;
            rank[b] = 0;
        }
        for (int e = 0; e < E; ++e) {
            int base = 0;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (32 * b >= n)
                    break;
                const uint32_t hit = __ballot_sync(0xffffffffu, v[b] == e);
                if (v[b] == e)
                    rank[b] = base + __popc(hit & ((1u << lane) - 1));
                base += __popc(hit);
            }
            cnt = lane == e ? base : cnt;
        }
        const int kept = a.C < 0 ? cnt : min(cnt, a.C);
        int off = kept;  // inclusive prefix sum
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, off, o);
            off += lane >= o ? u : 0;
        }
        const uint32_t used = __ballot_sync(0xffffffffu, kept > 0);
        if (lane < E) {
            s_cnt[lane] = cnt;
            s_kept[lane] = kept;
            s_off[lane + 1] = off;
            if (kept > 0)
                s_sel[__popc(used & ((1u << lane) - 1))] = lane;
        }
        if (lane == 0) {
            s_off[0] = 0;
            s_nsel = __popc(used);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (32 * b >= n)
                break;
            const int e = max(v[b], 0), i = 32 * b + lane;
            const int first = __shfl_sync(0xffffffffu, off - kept, e);
            const int room = __shfl_sync(0xffffffffu, kept, e);
            const int row = v[b] >= 0 && rank[b] < room ? first + rank[b] : -1;
            if (i < n)
                s_slot[i] = row;
            if (row >= 0)
                s_rtok[row] = i / k;
        }
    } else if (one_window) {
        stage_rows<true>(region, pitch1, s_inv, T, 0, chunks1, d, nullptr, 0, 1);
    }
    __syncthreads();
    const int nsel = s_nsel, R = s_off[E], m8 = round_up(m, 8);
    uint32_t a_off[4];  // this lane's words of A row g in a chunk
#pragma unroll
    for (int b = 0; b < 4; ++b)
        a_off[b] = (uint32_t)(g * 64 + ((b ^ ((g >> 1) & 3)) << 4) + c * 4);

    // ---- one product phase over the table's items: their sums, handed to done(item, slot,
    // sum) for PER slots an item, where sum(L, q) is value q of lane L.  A group's warps add
    // their parts in warp order; groups wait for one another only to stage a window.
    auto products = [&](auto &ph, auto &ld, auto per, int pitch, bool staged, auto stage, auto brow,
                        auto done) {
        constexpr int PER = decltype(per)::value;
        const int grp = ph.group(), nks = 1 << ph.kshift, ks = warp & (nks - 1);
        uint32_t st = ring_s;
        float *part = red;  // two buffers in turn: one barrier an item
        int buf = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < ph.n_items; i0 += ph.groups()) {
            const int i = i0 + grp;
            const bool mine = i < ph.n_items;
            const int32_t item = ph.items[mine ? i : 0];
            float acc[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[nb][q] = 0.f;
#pragma unroll 1
            for (int w = 0; w < ph.n_win; ++w) {
                if (!staged || ph.n_win > 1) {
                    if (i0 + w > 0)
                        __syncthreads();  // the last window's products are done
                    stage(w);
                    __syncthreads();
                    staged = true;
                }
                if (!mine)
                    continue;
                int lo, hi;
                ph.share(w, lo, hi);
                const int chunks = ph.chunks(w);
                uint32_t bp[NB], ip[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    bp[nb] = region_s + (uint32_t)(brow(item, nb * 8 + g) * pitch +
                                                   lo * stage_cols(NB) * 2 + 16 * c);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        ip[nb][j] = smem_u32(s_inv + brow(item, nb * 8 + 2 * c + j) * chunks + lo * SC);
                }
#pragma unroll 1
                for (int n = hi - lo; n > 0; --n) {
                    __syncwarp();  // the stage the loader fills next has been read
                    ld.issue();
                    cp_wait<DEPTH - 1>();
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < SC; ++u) {
                        chunk_mma<NB>(acc, st + u * kChunkBytes, a_off, bp, ip, g);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            bp[nb] += kChunkCols * 2;
                            ip[nb][0] += 4;
                            ip[nb][1] += 4;
                        }
                    }
                    st = st + SB == ring_s + DEPTH * SB ? ring_s : st + SB;
                }
            }
            if (!mine)
                continue;
            float *rw = part + ((size_t)(buf * kWarps + warp) * 32 + lane) * RQ;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    rw[nb * 4 + q] = acc[nb][q];
            if (ph.kshift == 0)
                __syncwarp();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(32 << ph.kshift) : "memory");
            const float *r0 = part + (size_t)(buf * kWarps + (grp << ph.kshift)) * 32 * RQ;
#pragma unroll 1
            for (int j = ks * 32 + lane; j < PER; j += 32 << ph.kshift)
                done(item, j, [&](int L, int q) {
                    const float *r = r0 + (size_t)L * RQ + q;
                    float v = 0.f;
#pragma unroll 4
                    for (int u = 0; u < nks; ++u)
                        v += r[(size_t)u * 32 * RQ];
                    return v;
                });
            buf ^= 1;
        }
    };

    // ---- GEMM 1
    const UpItems up(nsel, m);
    const int n_up = up.hi > up.lo ? up.count() : 0;
#pragma unroll 1
    for (int base = 0; base < n_up; base += kItems) {
        Phase<true, NB> ph(a, s_items);
        ph.set(min(kItems, n_up - base));
        if (base > 0)
            __syncthreads();  // the table's last use is over
        if ((int)threadIdx.x < ph.n_items) {
            int is, q, n;
            up.get(base + threadIdx.x, is, q, n);
            s_items[threadIdx.x] = item_pack(s_sel[is], q, n);
        }
        __syncthreads();
        Loader<true, NB, DEPTH> ld(ph, ring_s);
        products(
            ph, ld, std::integral_constant<int, 64 * NB>(), pitch1, one_window,
            [&](int w) {
                stage_rows<false>(region, pitch1, s_inv, T, w * a.win1, ph.chunks(w), d, a.x, d, 0);
            },
            [&](int32_t item, int tok) {
                const int e = item_expert(item), r0 = s_off[e];
                return s_rtok[min(r0 + tok, s_off[e + 1] - 1)];
            },
            [&](int32_t item, int slot, auto sum) {
                const int e = item_expert(item), r0 = s_off[e], nr = s_off[e + 1] - r0;
                const int s = slot & 7, tok = slot >> 3;
                const int nrn = up_neuron(item_first(item), s);
                const int L = s * 4 + (tok & 7) / 2, at = tok / 8 * 4 + (tok & 1);
                if (s < 4 * item_quads(item) && nrn < m && tok < nr) {
                    const float gv = sum(L, at), uv = sum(L, at + 2);
                    // approximate division (2 ulp, 0 once 1 + e^-g > 2^126, silu's limit)
                    a.h[(int64_t)(r0 + tok) * m8 + nrn] =
                        __float2bfloat16_rn(__fdividef(gv, 1.0f + __expf(-gv)) * uv);
                }
            });
    }

    // ---- h of every CTA complete: a grid barrier; GEMM 2's first weights travel meanwhile,
    // and CTA 0 writes the routing, the tables and the statistics
    const DownItems down(d);
    const int n_down = nsel * down.per;
    Phase<false, NB> ph(a, s_items);
    auto fill_down = [&](int base) {
        ph.set(min(kItems, n_down - base));
        if ((int)threadIdx.x < ph.n_items) {
            int is, q, n;
            down.get(base + threadIdx.x, is, q, n);
            s_items[threadIdx.x] = item_pack(s_sel[is], q, n);
        }
    };
    __syncthreads();  // h of this CTA is written, the table's last use is over
    if (threadIdx.x == kThreads - 1) {
        __threadfence();  // this CTA's h, ordered before by the barrier above
        if (atomicAdd(a.gbar, 1) == (int)gridDim.x - 1) {  // the last to arrive releases all
            __threadfence();
            asm volatile("red.relaxed.gpu.global.and.b32 [%0], 0;" ::"l"(a.gbar) : "memory");
            __threadfence();
            atomicAdd(a.gbar + 1, 1);
        }
    }
    fill_down(0);
    __syncthreads();
    Loader<false, NB, DEPTH> ld(ph, ring_s);
    if (threadIdx.x == 0) {
        const uint64_t t0 = globaltimer_ns();
        while (ld_acquire_gpu(a.gbar + 1) == gen) {
            if (globaltimer_ns() - t0 > a.wait_ns) {
                set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                s_abort = 1;
                break;
            }
        }
    } else if (blockIdx.x == 0 && threadIdx.x >= 32) {
        constexpr int nt = kThreads - 32;
        const int t1 = (int)threadIdx.x - 32;
        if (t1 < T * k) {
            a.idx[t1] = s_idx[t1];
            a.w[t1] = s_w[t1];
            a.slot_row[t1] = s_slot[t1];
        }
        if (t1 < R)
            a.row_token[t1] = s_rtok[t1];
        if (t1 <= E)
            a.offsets[t1] = s_off[t1];
        // the gate statistics, in gate_stats_kernel's arithmetic
        if (t1 < E) {
            float sp = 0.f, sg = 0.f;
            for (int t = 0; t < T; ++t) {
                sp += s_prob[t * E + t1];
                sg += s_gw[t * E + t1];
            }
            a.counts[t1] = s_cnt[t1];
            a.kept[t1] = s_kept[t1];
            a.probs_sum[t1] = sp;
            a.importance[t1] = sg;
            a.f[t1] = (float)((double)s_cnt[t1] / ((double)T * k));
            a.P[t1] = (float)((double)sp / (double)T);
        }
        if (t1 == nt - 1) {
            double sfp = 0.0;
            for (int e = 0; e < E; ++e) {
                float sp = 0.f;
                for (int t = 0; t < T; ++t)
                    sp += s_prob[t * E + e];
                sfp += ((double)s_cnt[e] / ((double)T * k)) * ((double)sp / (double)T);
            }
            a.loss[0] = (float)(a.lambda * sfp);
        }
    }
    __syncthreads();

    // ---- GEMM 2 and the combine of this CTA's columns
    if (!s_abort) {
        const int ncol = 4 * (down.hi - down.lo);
#pragma unroll 1
        for (int base = 0; base < n_down;) {
            products(
                ph, ld, std::integral_constant<int, 128 * NB>(), pitch2, base > 0,
                [&](int w) {
                    stage_rows<false>(region, pitch2, s_inv, R, w * a.win2, ph.chunks(w), m, a.h,
                                      m8, 0);
                },
                [&](int32_t item, int tok) {
                    const int e = item_expert(item);
                    return min(s_off[e] + tok, s_off[e + 1] - 1);
                },
                [&](int32_t item, int slot, auto sum) {
                    const int e = item_expert(item), r0 = s_off[e], nr = s_off[e + 1] - r0;
                    const int s = slot & 15, tok = slot >> 4;
                    const int L = (s & 7) * 4 + (tok & 7) / 2;
                    const int at = tok / 8 * 4 + (tok & 1) + (s & 8) / 4;
                    if (s < 4 * item_quads(item) && tok < nr)
                        outs[(size_t)(r0 + tok) * ncol + 4 * (item_first(item) - down.lo) + s] =
                            sum(L, at);
                });
            base += kItems;
            if (base < n_down) {
                __syncthreads();
                fill_down(base);
                __syncthreads();
                ld.restart();
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < T * ncol; i += kThreads) {
            const int t = i / ncol, o = i - t * ncol;
            const int col = down_column(down.lo, o);
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
    cp_wait<0>();
}

// --------------------------------------------------------------------- host side

constexpr int kDepths = 3;
constexpr int kDepth[kDepths] = {4, 3, 2};  // stages of a warp's ring
typedef void (*Kernel)(const Args);
static const Kernel kKernel[2][kDepths] = {
    {mx4_few_kernel<1, 4>, mx4_few_kernel<1, 3>, mx4_few_kernel<1, 2>},
    {mx4_few_kernel<2, 4>, mx4_few_kernel<2, 3>, mx4_few_kernel<2, 2>}};

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
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return e;
        for (int i = 0; i < 2 * kDepths; ++i)
            if ((e = cudaFuncSetAttribute(kKernel[i / kDepths][i % kDepths],
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)kSmemCap)) != cudaSuccess)
                return e;
        sms[dev] = n;
    }
    *out = sms[dev];
    return cudaSuccess;
}

// Columns staged at once for `rows` activation rows of K columns: all of them if they fit
// the region and the table of scales, else as many whole chunks as do.
static int window(int rows, int K, int nb)
{
    const int unit = stage_cols(nb), all = (K + unit - 1) / unit * unit;
    int w = (kMaxRegion / rows - 64) / 2;
    const int t = kMaxInv / rows * kChunkCols;
    w = w < t ? w : t;
    w = (w < kMaxWindow ? w : kMaxWindow) / unit * unit;
    return w < all ? w : all;
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
    a.win1 = window(p->T, p->d, nb);
    a.win2 = window(R, p->m, nb);
    const int x_bytes = p->T * row_pitch(a.win1), h_bytes = R * row_pitch(a.win2);
    a.region = round_up(x_bytes > h_bytes ? x_bytes : h_bytes, 128);
    // two buffers of the warps' sums; the router's partial logits come there first
    const int part = kWarps * p->T * round_up((b->Wnoise != nullptr ? 2 : 1) * p->E, 8) * 4;
    a.red = 2 * kWarps * 32 * 4 * nb * 4;
    a.red = round_up(a.red > part ? a.red : part, 128);
    const int64_t quads = (p->d + 127) / 128 * 32;
    const size_t outs = (size_t)R * 4 * ((quads + grid - 1) / grid + 1) * 4;
    const size_t fixed = (size_t)a.region + a.red + outs, per = (size_t)kWarps * stage_bytes(nb);
    int di = 0;
    while (di < kDepths && fixed + kDepth[di] * per > kSmemCap)
        ++di;
    if (di == kDepths)
        return cudaErrorInvalidValue;
    const size_t smem = fixed + kDepth[di] * per;
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
    e = cudaLaunchKernelEx(&cfg, kKernel[nb - 1][di], a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace moe
