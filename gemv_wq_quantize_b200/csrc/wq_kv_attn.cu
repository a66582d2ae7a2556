// wq_kv_attn.cu -- kv_attention: the C entry points, and the kernel for few rows per key head
// (decode and draft verification): attention over the paged 8-bit cache, split over the whole
// GPU by key ranges.
//
// Mathematics: for a query row q of position p and the keys j <= p of its sequence,
//   s_j = sm_scale * ks[page(j)] * (q . kc_j),   out = sum_j softmax(s)_j vs[page(j)] vc_j
// with the codes kc, vc exact in binary16, products on mma.sync with binary32 accumulation, one
// pass with a running maximum and sum, and the two page scales applied in binary32.
//
// Bound by reading the cache once.  A group of query heads shares a key head's codes, so the rows
// of (sequence, key head) form the 8-wide N side of both products (S^T = K Q^T and
// O^T = V^T P^T): the codes are the 16-row A operand and nothing is wasted on padding up to 8
// rows (an M side of 128 rows of tcgen05 would be 8 of 128 full).  Every warp walks its own keys
// with a small ring of its own: TMA copies of 32 keys or values (16 at head sizes above 128) into
// swizzled shared memory, the next ones issued by the warp as soon as it has read a buffer, so
// two are in flight while it multiplies a third and no warp waits for another between the ends of
// a tile.  The swizzle makes the fragment reads free of bank conflicts; a dot product may take its
// dimensions in any order, so a lane's 16 contiguous bytes of a key are its fragments of four MMA
// steps, and its 16 contiguous bytes of four values are its fragments of eight row tiles.
//
// Work split: tiles (sequence, key head, 8 * NT rows) are cut into units of 64 keys, and the
// persistent blocks take equal contiguous shares of all units, whatever the lengths (a tile counts
// kTileUnits more, about what its start and end take).  A tile cut over several blocks leaves
// partial sums in the workspace; the last block to arrive adds them in the order of their keys,
// so the result does not depend on which block that is.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "wq_act.cuh"
#include "wq_kv_attn.cuh"

namespace wq {

static __device__ int g_kv_attn_error;

int kv_attn_read_error()
{
    int v = 0, zero = 0;
    cudaMemcpyFromSymbol(&v, g_kv_attn_error, sizeof v);
    cudaMemcpyToSymbol(g_kv_attn_error, &zero, sizeof zero);
    return v;
}

namespace {

constexpr int kWarps = 6;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnitShift = 6;     // a unit: 64 keys, the granule of the split
constexpr int kTileUnits = 6;     // what the start and end of a tile cost a block, in units
constexpr int kLeastUnits = 4;    // of a share: a stage for each warp; less only adds partials
constexpr int kMostUnits = 1 << 30;

// exp2 arguments are raised by 15: the weights then reach 2^15 in binary16 (its largest is just
// below 2^16) and keep full precision down to 2^-29 of the largest weight, so that many small
// weights under one large one are not lost; the sum carries the same factor.
constexpr float kRaise = 15.f;

__device__ __forceinline__ uint32_t trans8x8(uint32_t x)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}

__device__ __forceinline__ uint64_t globaltimer()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// DT: head_dim rounded up to 64, 128 or 256.  NT: tiles of 8 rows.
template <int DT, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kPerSm = DT <= 128 && NT == 1 ? 2 : 1;  // blocks: 128 or 255 registers a thread
    static constexpr int kSteps = DT <= 128 ? 2 : 1;             // 16-key steps of a stage
    static constexpr int kKeys = 16 * kSteps;
    static constexpr int kRowBytes = DT < 128 ? 64 : 128;        // of a copied box; two boxes at DT 256
    static constexpr int kBoxes = DT / 128 < 1 ? 1 : DT / 128;
    static constexpr int kBoxBytes = kKeys * kRowBytes;
    static constexpr int kItem = kBoxBytes * kBoxes;             // the keys (or values) of a stage
    static constexpr int kBufs = kPerSm == 2 ? 4 : 5;            // items of a warp's ring
    static constexpr int kRowFloats = DT + 4;                    // a partial row: sums, maximum, weight sum
};

// A row of sums in shared memory and in the workspace is kept in the order of the fragments:
// place 16 i + 2 g + e holds dimension dim_of(that) (lane (g, j) then stores pairs without bank
// conflicts, rows being DT + 4 apart).
template <int DT>
__device__ __forceinline__ int dim_of(int place)
{
    const int i = place / 16, g = place % 16 / 2, e = place % 2;
    return DT == 64 ? 8 * g + 2 * i + e : 128 * (i / 8) + 16 * g + 2 * (i % 8) + e;
}

template <int DT, int NT>
struct Smem {
    using S = Shape<DT, NT>;
    alignas(1024) uint8_t ring[kWarps][S::kBufs][S::kItem];
    uint64_t full[kWarps][S::kBufs];
    float o[kWarps][8 * NT][DT / 4 + 4];   // a quarter of the warps' sums at a time
    float m[kWarps][8 * NT], l[kWarps][8 * NT], f[kWarps][8 * NT];
    float top[8 * NT], weight[8 * NT];     // of a row over the warps
    int64_t sums[kWarps];
    int first[2], parts[2];                // the tiles that this block left partials of
    int abort;
    // then the unit counts of all sequences up to each (n_seqs + 1)
};

// A bounded wait with one answer for the warp: about 2 s, or 20 ms once another warp gave up.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    bool ok = false;
    for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait_short(bar, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer();
        while (!ok) {
            for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait_short(bar, parity);
            if (!ok && globaltimer() - t0 > (*abort ? 20000000ull : 2000000000ull)) {
                atomicCAS(&g_kv_attn_error, kErrNone, kErrWaitTimeout);
                *abort = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// The codes of 16 keys of a stage in the registers of a warp, from swizzled shared memory.
// Keys: lane (g, j) has keys g and g + 8, dimensions kdim(c, j) .. + 15.
template <int DT>
__device__ __forceinline__ int kdim(int c, int j)
{
    return DT == 64 ? 16 * j : 128 * (c / 2) + 32 * j + 16 * (c % 2);
}
template <int DT, int NT>
__device__ __forceinline__ uint4 key_chunk(const uint8_t *k, int row, int c, int j)
{
    if constexpr (DT == 64) return lds128(k + row * 64 + ((j ^ ((row >> 1) & 3)) << 4));
    else return lds128(k + c / 2 * Shape<DT, NT>::kBoxBytes + row * 128 + (((2 * j + c % 2) ^ (row & 7)) << 4));
}
// Values: lane (g, j) has keys 2j, 2j + 1, 2j + 8, 2j + 9 and DT / 8 bytes of each.
template <int DT, int NT>
__device__ __forceinline__ void value_words(const uint8_t *v, int row, int g, uint32_t (&w)[DT / 32])
{
    if constexpr (DT == 64) {
        const uint2 x = lds64(v + row * 64 + (((g / 2) ^ ((row >> 1) & 3)) << 4) + 8 * (g % 2));
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int c = 0; c < DT / 128; ++c) {
            const uint4 x = lds128(v + c * Shape<DT, NT>::kBoxBytes + row * 128 + ((g ^ (row & 7)) << 4));
            w[4 * c] = x.x;
            w[4 * c + 1] = x.y;
            w[4 * c + 2] = x.z;
            w[4 * c + 3] = x.w;
        }
    }
}

// One warp's running state over its keys: column n of the products is row n of the tile.
template <int DT, int NT>
struct State {
    float o[NT][DT / 16][4];  // lane (g, j): places 16 i + 2 g and + 1; rows 2j, 2j + 1
    float m[NT][2], l[NT][2];
};

// Queries as B fragments (binary16): k-step 4 c + w holds, for lane (g, j) and row g, the
// dimensions kdim(c, j) + 4 w .. + 3.  A bfloat16 row is scaled by a power of two so that its
// largest value fits binary16; what falls below the smallest subnormal there is under 2^-25 of
// the row's largest value, the size of the binary32 accumulation's own rounding.  The scale's
// inverse comes back for rows 2j and 2j + 1.
template <bool BF16, int DT, int NT>
__device__ __forceinline__ void load_queries(const KvAttnArgs &a, const KvSpan &s, int head, int row0, int rows, int g,
                                             int j, uint32_t (&qf)[NT][DT / 16][2], float (&unscale)[NT][2])
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + g;
        const bool live = 8 * n + g < rows;
        const int i = live ? r / a.group : 0, h = live ? r % a.group : 0;
        const uint16_t *q = static_cast<const uint16_t *>(a.q) +
                            (int64_t(s.q0 + i) * a.q_heads + head * a.group + h) * a.head_dim;
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < DT / 64; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int d = kdim<DT>(c, j) + 4 * w;
                const uint2 x = live && d < a.head_dim ? *reinterpret_cast<const uint2 *>(q + d) : make_uint2(0, 0);
                qf[n][4 * c + w][0] = x.x;
                qf[n][4 * c + w][1] = x.y;
                if constexpr (BF16) {
                    const float2 lo = act_f2<__nv_bfloat16>(x.x), hi = act_f2<__nv_bfloat16>(x.y);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(lo.x), fabsf(lo.y)), fmaxf(fabsf(hi.x), fabsf(hi.y))));
                }
            }
        unscale[n][0] = unscale[n][1] = 1.f;
        if constexpr (BF16) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^-e with e the exponent of the largest value: the row's values stay within 2
            const int e = kv_clamp(int(__float_as_uint(amax) >> 23) - 127, -120, 120);
            const float up = __uint_as_float(uint32_t(127 - e) << 23), down = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < DT / 16; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 v = act_f2<__nv_bfloat16>(qf[n][k][x]);
                    qf[n][k][x] = act_t2<__half>(v.x * up, v.y * up);
                }
            unscale[n][0] = __shfl_sync(0xffffffffu, down, 8 * j);       // row 2j is lane (2j, 0)
            unscale[n][1] = __shfl_sync(0xffffffffu, down, 8 * j + 4);
        }
    }
}

// Scores of 16 keys (rows row0 .. + 15 of a stage): S^T[key][row], lane (g, j) holds keys g and
// g + 8, rows 2j and 2j + 1.
template <bool F8, int DT, int NT>
__device__ __forceinline__ void scores(const uint8_t *k, int row0, int g, int j, const uint32_t (&qf)[NT][DT / 16][2], float (&s)[NT][4])
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
    for (int c = 0; c < DT / 64; ++c) {
        const uint4 r0 = key_chunk<DT, NT>(k, row0 + g, c, j), r1 = key_chunk<DT, NT>(k, row0 + g + 8, c, j);
        const uint32_t lo[4] = {r0.x, r0.y, r0.z, r0.w}, hi[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t x = F8 ? lo[w] : lo[w] ^ 0x80808080u, y = F8 ? hi[w] : hi[w] ^ 0x80808080u;
            const uint32_t f[4] = {widen<F8, 0>(x), widen<F8, 0>(y), widen<F8, 1>(x), widen<F8, 1>(y)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(s[n], f, qf[n][4 * c + w][0], qf[n][4 * c + w][1]);
        }
    }
}

// O^T += vs * (V^T P^T) over 16 keys; p: the weights as B fragments.  left: keys of the 16 that
// hold codes (the slots behind may hold e4m3 NaN codes).
template <bool F8, int DT, int NT>
__device__ __forceinline__ void add_values(const uint8_t *v, int row0, int left, int g, int j,
                                           const uint32_t (&p)[NT][2], float vs, State<DT, NT> &st)
{
    uint32_t w[4][DT / 32];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int key = 2 * j + (t & 1) + 8 * (t >> 1);
        value_words<DT, NT>(v, row0 + key, g, w[t]);
        if (F8 && left < 16 && key >= left)
#pragma unroll
            for (int x = 0; x < DT / 32; ++x) w[t][x] = 0u;
    }
#pragma unroll
    for (int i = 0; i < DT / 16; i += 2) {
        // bytes 2i .. 2i + 3 of the lane's chunk of four keys: row tiles i and i + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t a = prmt(w[0][i / 2], w[1][i / 2], e ? 0x7362 : 0x5140);
            uint32_t b = prmt(w[2][i / 2], w[3][i / 2], e ? 0x7362 : 0x5140);
            if constexpr (!F8) {
                a ^= 0x80808080u;
                b ^= 0x80808080u;
            }
            const uint32_t f[4] = {widen<F8, 0>(a), widen<F8, 1>(a), widen<F8, 0>(b), widen<F8, 1>(b)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(acc, f, p[n][0], p[n][1]);
#pragma unroll
                for (int x = 0; x < 4; ++x) st.o[n][i + e][x] = fmaf(vs, acc[x], st.o[n][i + e][x]);
            }
        }
    }
}

struct Tile {
    KvSpan s;
    int b, head, row0, rows;
    int keys;      // keys that the tile's last row sees
    int t0, t1;    // keys of this block's units of the tile
    int u0, u1;    // units of the tile, counted over all sequences: the first that holds keys, the end
    bool first;    // this block's part begins the tile's keys, and
    bool whole;    // ends them
};

// The tile of unit u and this block's part of it (units up to u_end); next: the unit behind it.
// A part without keys (of a tile's first kTileUnits units alone) has t1 = t0 and is passed over,
// but for the first part of a tile that has none at all.
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const KvAttnArgs &a, const int *before, int shift, int u, int u_end, int &next)
{
    // the sequence of unit u: the last b with before[b] <= u (empty ones have no units)
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (before[mid] <= u) lo = mid;
        else hi = mid;
    }
    Tile t;
    t.b = lo;
    t.s = kv_span(__ldg(a.cu_q + lo), __ldg(a.cu_q + lo + 1), __ldg(a.seq_len + lo), a.M, a.capacity);
    const bool split = a.partials != nullptr;
    const int head_units = split ? kTileUnits : 0;
    const int units = split ? head_units + int(kv_units(t.s.len, 1 << shift)) : 1;
    const int tiles = (t.s.n * a.group + ROWS - 1) / ROWS;
    const int item = (u - before[lo]) / units;  // (key head, tile) of the sequence
    const int begin = before[lo] + item * units, end = begin + units;
    next = min(end, u_end);
    t.head = item / tiles;
    t.row0 = item % tiles * ROWS;
    t.rows = min(ROWS, t.s.n * a.group - t.row0);
    t.keys = max(0, t.s.len - t.s.n + (t.row0 + t.rows - 1) / a.group + 1);
    t.u0 = begin + head_units;
    t.u1 = end;
    if (split) {
        t.t0 = int(min(int64_t(t.keys), int64_t(max(0, u - t.u0)) << shift));
        t.t1 = int(min(int64_t(t.keys), int64_t(max(0, next - t.u0)) << shift));
    } else {
        t.t0 = 0;
        t.t1 = t.keys;
    }
    t.first = u <= t.u0 && next > t.u0;
    t.whole = t.first && next == end;
    return t;
}

// A warp's walk over its stages of a tile (every kWarps-th) with its ring of items (keys and values
// of its stages in turn).  begin() looks up the pages and sends for the first items; run() takes
// them in.  Between the two a block joins the sums of its tile before, while the copies travel.
template <int DT, int NT>
struct Walk {
    using S = Shape<DT, NT>;
    struct Pages {  // lane l has those of the warp's stage base + l
        int z[2];   // (page, head) of the stage's boxes; -1: none; -2: no page
        float ks[S::kSteps], vs[S::kSteps];
    };
    const KvAttnArgs &a;
    const CUtensorMap *km, *vm;
    Smem<DT, NT> &sm;
    Tile t;
    Pages cur, next;
    int mine;        // the warp's stages: warp + i * kWarps
    int base;        // the stage that lane 0's pages are for
    int issued;      // items
    uint32_t item0;  // items of the warp over all tiles before: item x goes to buffer (item0 + x) % kBufs

    __device__ __forceinline__ Walk(const KvAttnArgs &a_, const CUtensorMap *km_, const CUtensorMap *vm_, Smem<DT, NT> &sm_)
        : a(a_), km(km_), vm(vm_), sm(sm_), mine(0), item0(0)
    {
    }
    __device__ __forceinline__ int box_rows() const { return min(1 << a.page_shift, S::kKeys); }
    __device__ __forceinline__ bool two() const { return (1 << a.page_shift) < S::kKeys; }  // a stage lies in two pages
    __device__ __forceinline__ int key_of(int i) const { return t.t0 + (int(threadIdx.x) / 32 + i * kWarps) * S::kKeys; }

    __device__ __forceinline__ void look_up(Pages &p, int i)
    {
        const int32_t *table = a.block_table + int64_t(t.b) * a.max_pages;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int key = key_of(i) + x * 16;
            p.z[x] = -1;
            if (i < mine && key < t.t1 && (x == 0 || two())) {
                const int64_t page = kv_page_ok(__ldg(table + (key >> a.page_shift)), a.num_pages);
                p.z[x] = page < 0 ? -2 : int(page) * a.kv_heads + t.head;
            }
        }
    }
    __device__ __forceinline__ void look_up_scales(Pages &p)
    {
#pragma unroll
        for (int e = 0; e < S::kSteps; ++e) {
            const int z = two() && e ? p.z[1] : p.z[0];
            p.ks[e] = z >= 0 ? __ldg(a.k_scale + z) : 0.f;
            p.vs[e] = z >= 0 ? __ldg(a.v_scale + z) : 0.f;
        }
    }
    __device__ __forceinline__ void issue()
    {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        const int x = issued++, i = x / 2 - base;
        const int z0 = __shfl_sync(0xffffffffu, i < 32 ? cur.z[0] : next.z[0], i % 32);
        const int z1 = __shfl_sync(0xffffffffu, i < 32 ? cur.z[1] : next.z[1], i % 32);
        if (lane == 0) {
            const uint32_t b = (item0 + x) % S::kBufs;
            uint8_t *dst = sm.ring[warp][b];
            uint64_t *bar = &sm.full[warp][b];
            const CUtensorMap *map = x & 1 ? vm : km;
            const uint32_t bytes = uint32_t(box_rows() * S::kRowBytes * S::kBoxes);
            mbar_arrive_expect_tx(bar, (z0 >= 0 ? bytes : 0u) + (z1 >= 0 ? bytes : 0u));
            const int y = two() ? 0 : key_of(x / 2) & ((1 << a.page_shift) - 1);
#pragma unroll
            for (int c = 0; c < S::kBoxes; ++c) {
                if (z0 >= 0) tma_load_3d(dst + c * S::kBoxBytes, map, 128 * c, y, z0, bar);
                if (z1 >= 0) tma_load_3d(dst + c * S::kBoxBytes + 16 * S::kRowBytes, map, 128 * c, 0, z1, bar);
            }
            if (z0 == -2 || z1 == -2) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
        }
    }
    __device__ __forceinline__ bool ready(int x)
    {
        return wait_warp(&sm.full[threadIdx.x / 32][(item0 + x) % S::kBufs], ((item0 + x) / S::kBufs) & 1, &sm.abort);
    }

    // All items of the tile before are taken in (the ring is free).
    __device__ __forceinline__ void begin(const Tile &tile)
    {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        item0 += 2u * uint32_t(mine);
        t = tile;
        const int n = (t.t1 - t.t0 + S::kKeys - 1) / S::kKeys;  // stages of the tile
        mine = max(0, n - warp + kWarps - 1) / kWarps;
        base = issued = 0;
        if (mine == 0) return;
        look_up(cur, lane);
        look_up_scales(cur);  // in front of the copies, which would delay them
#pragma unroll 1
        while (issued < min(int(S::kBufs), 2 * mine)) issue();
        look_up(next, 32 + lane);
    }
    template <bool F8, bool BF16>
    __device__ __forceinline__ void run(State<DT, NT> &st);
};

template <int DT, int NT>
template <bool F8, bool BF16>
__device__ __forceinline__ void Walk<DT, NT>::run(State<DT, NT> &st)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, j = lane % 4;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
        st.m[r][0] = st.m[r][1] = -INFINITY;
        st.l[r][0] = st.l[r][1] = 0.f;
#pragma unroll
        for (int i = 0; i < DT / 16; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) st.o[r][i][x] = 0.f;
    }
    if (mine == 0) return;
    const int items = 2 * mine;
    uint32_t qf[NT][DT / 16][2];
    float qs[NT][2];
    load_queries<BF16, DT, NT>(a, t.s, t.head, t.row0, t.rows, g, j, qf, qs);
    int seen[NT][2];  // keys that rows 2j and 2j + 1 see
#pragma unroll
    for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int row = 8 * r + 2 * j + x;
            seen[r][x] = row < t.rows ? min(t.t1, t.s.len - t.s.n + (t.row0 + row) / a.group + 1) : 0;
            qs[r][x] *= a.sm_scale * kLog2e;
        }
    const int least = min(t.t1, t.s.len - t.s.n + t.row0 / a.group + 1);  // keys that every row sees

    const bool pair = two();
    int done = 0;  // items waited for
    for (int i = 0; i < mine; ++i) {
        if (i - base == 32) {
            base += 32;
            cur = next;
            look_up(next, base + 32 + lane);
        }
        if (i - base == 8) look_up_scales(next);
        const int key = key_of(i);
        float s[S::kSteps][NT][4], vs[S::kSteps];
        const uint8_t *k = sm.ring[warp][(item0 + 2 * i) % S::kBufs], *v = sm.ring[warp][(item0 + 2 * i + 1) % S::kBufs];
        if (!ready(done++)) break;
#pragma unroll
        for (int e = 0; e < S::kSteps; ++e) {
            scores<F8, DT, NT>(k, 16 * e, g, j, qf, s[e]);
            const float ks = __shfl_sync(0xffffffffu, cur.ks[e], i - base);
            vs[e] = __shfl_sync(0xffffffffu, cur.vs[e], i - base);
            const int z = __shfl_sync(0xffffffffu, pair && e ? cur.z[1] : cur.z[0], i - base);
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[e][r][x] *= ks * qs[r][x & 1];
            const int first = key + 16 * e;
            if (first + 16 > least || z < 0) {
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (first + g + 8 * (x >> 1) >= seen[r][x & 1] || z < 0) s[e][r][x] = -INFINITY;
            }
        }
        __syncwarp();  // the keys are read: their buffer takes the next item
        if (issued < items) issue();
        uint32_t p[S::kSteps][NT][2];
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            float mx[2] = {st.m[r][0], st.m[r][1]};
#pragma unroll
            for (int e = 0; e < S::kSteps; ++e)
#pragma unroll
                for (int x = 0; x < 4; ++x) mx[x & 1] = fmaxf(mx[x & 1], s[e][r][x]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
            }
            if (__any_sync(0xffffffffu, mx[0] > st.m[r][0] || mx[1] > st.m[r][1])) {
                // -inf - -inf: no key seen yet, nothing to rescale
                const float f0 = mx[0] == st.m[r][0] ? 1.f : exp2_approx(st.m[r][0] - mx[0]);
                const float f1 = mx[1] == st.m[r][1] ? 1.f : exp2_approx(st.m[r][1] - mx[1]);
                st.l[r][0] *= f0;
                st.l[r][1] *= f1;
#pragma unroll
                for (int c = 0; c < DT / 16; ++c) {
                    st.o[r][c][0] *= f0;
                    st.o[r][c][1] *= f1;
                    st.o[r][c][2] *= f0;
                    st.o[r][c][3] *= f1;
                }
                st.m[r][0] = mx[0];
                st.m[r][1] = mx[1];
            }
            const float low[2] = {mx[0] == -INFINITY ? 0.f : mx[0] - kRaise, mx[1] == -INFINITY ? 0.f : mx[1] - kRaise};
#pragma unroll
            for (int e = 0; e < S::kSteps; ++e) {
                float w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    w[x] = exp2_approx(s[e][r][x] - low[x & 1]);
                    st.l[r][x & 1] += w[x];
                }
                // weights to binary16: half a step is 2^-12 of each, of either sign
                p[e][r][0] = trans8x8(act_t2<__half>(w[0], w[1]));
                p[e][r][1] = trans8x8(act_t2<__half>(w[2], w[3]));
            }
        }
        if (!ready(done++)) break;
#pragma unroll
        for (int e = 0; e < S::kSteps; ++e) {
            const int z = __shfl_sync(0xffffffffu, pair && e ? cur.z[1] : cur.z[0], i - base);
            add_values<F8, DT, NT>(v, 16 * e, z < 0 ? 0 : t.t1 - (key + 16 * e), g, j, p[e], vs[e], st);
        }
        __syncwarp();
        if (issued < items) issue();
    }
    // (only after a wait gave up: nothing may land in memory that is used for something else)
    while (done < issued) ready(done++);
}

__device__ __forceinline__ uint16_t *out_row(const KvAttnArgs &a, const Tile &t, int r)
{
    const int row = t.row0 + r;
    return static_cast<uint16_t *>(a.out) +
           (int64_t(t.s.q0 + row / a.group) * a.q_heads + t.head * a.group + row % a.group) * a.head_dim;
}
__device__ __forceinline__ float inverse_of(float l) { return l > 0.f ? 1.f / l : (l == l ? 0.f : l); }
__device__ __forceinline__ float weight_of(float m, float top) { return m == -INFINITY ? 0.f : exp2_approx(m - top); }

// The warps' states of a tile joined, a quarter of the places at a time: finished rows, or this
// block's partial in `slot`.
template <typename T, int DT, int NT>
__device__ __forceinline__ void join(const KvAttnArgs &a, Smem<DT, NT> &sm, const Tile &t, State<DT, NT> &st, float *slot)
{
    using S = Shape<DT, NT>;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, j = lane % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
            st.l[n][0] += __shfl_xor_sync(0xffffffffu, st.l[n][0], o);
            st.l[n][1] += __shfl_xor_sync(0xffffffffu, st.l[n][1], o);
        }
        if (g == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                sm.m[warp][8 * n + 2 * j + x] = st.m[n][x];
                sm.l[warp][8 * n + 2 * j + x] = st.l[n][x];
            }
        }
    }
    constexpr int kQuarter = DT / 4, kPairs = kQuarter / 2;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < DT / 64; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    *reinterpret_cast<float2 *>(&sm.o[warp][8 * n + 2 * j + x][16 * i + 2 * g]) =
                        make_float2(st.o[n][h * (DT / 64) + i][x], st.o[n][h * (DT / 64) + i][2 + x]);
        __syncthreads();
        if (h == 0) {
            if (tid < S::kRows) {
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][tid]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = weight_of(sm.m[w][tid], m);
                    sm.f[w][tid] = f;
                    l += f * sm.l[w][tid];
                }
                sm.top[tid] = m;
                sm.weight[tid] = l;
                if (slot && tid < t.rows) *reinterpret_cast<float2 *>(slot + tid * S::kRowFloats + DT) = make_float2(m, l);
            }
            __syncthreads();
        }
        for (int e = tid; e < t.rows * kPairs; e += kThreads) {
            const int r = e / kPairs, at = 2 * (e % kPairs), place = h * kQuarter + at;
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 v = *reinterpret_cast<const float2 *>(&sm.o[w][r][at]);
                x += sm.f[w][r] * v.x;
                y += sm.f[w][r] * v.y;
            }
            if (slot) {
                *reinterpret_cast<float2 *>(slot + r * S::kRowFloats + place) = make_float2(x, y);
            } else {
                const float inv = inverse_of(sm.weight[r]);
                const int d = dim_of<DT>(place);
                if (d < a.head_dim) *reinterpret_cast<uint32_t *>(out_row(a, t, r) + d) = act_t2<T>(x * inv, y * inv);
            }
        }
        __syncthreads();
    }
}

// Joins the partials of a tile: those of `parts` blocks from p0 on (its second slot, the others'
// first), in the order of their keys.
template <typename T, int DT, int NT>
__device__ __forceinline__ void join_parts(const KvAttnArgs &a, const Tile &t, const float *p0, int parts)
{
    using S = Shape<DT, NT>;
    constexpr int kQuads = DT / 4, kSlot = S::kRows * S::kRowFloats;
    constexpr int kBatch = 8;  // parts whose loads are in flight together
#pragma unroll 1
    for (int e = threadIdx.x; e < t.rows * kQuads; e += kThreads) {
        const int r = e / kQuads, place = 4 * (e % kQuads);
        float m = -INFINITY, l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int c0 = 0; c0 < parts; c0 += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int c = min(c0 + i, parts - 1);
                const float *row = p0 + c * (2 * kSlot) + (c == 0 ? kSlot : 0) + r * S::kRowFloats;
                ml[i] = __ldcg(reinterpret_cast<const float2 *>(row + DT));
                v[i] = __ldcg(reinterpret_cast<const float4 *>(row + place));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (c0 + i >= parts) break;
                const float top = fmaxf(m, ml[i].x), f = weight_of(m, top), w = weight_of(ml[i].x, top);
                l = f * l + w * ml[i].y;
                x.x = f * x.x + w * v[i].x;
                x.y = f * x.y + w * v[i].y;
                x.z = f * x.z + w * v[i].z;
                x.w = f * x.w + w * v[i].w;
                m = top;
            }
        }
        uint16_t *out = out_row(a, t, r);
        const float inv = inverse_of(l);
        const int d0 = dim_of<DT>(place), d1 = dim_of<DT>(place + 2);
        if (d0 < a.head_dim) *reinterpret_cast<uint32_t *>(out + d0) = act_t2<T>(x.x * inv, x.y * inv);
        if (d1 < a.head_dim) *reinterpret_cast<uint32_t *>(out + d1) = act_t2<T>(x.z * inv, x.w * inv);
    }
}

__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// kv_share in 32 bits (total and grid * grid fit).
__device__ __forceinline__ int share_of(int total, int c, int grid)
{
    const unsigned q = unsigned(total) / unsigned(grid), r = unsigned(total) % unsigned(grid);
    return int(q * unsigned(c) + r * unsigned(c) / unsigned(grid));
}

template <bool F8, bool BF16, int DT, int NT>
__device__ __forceinline__ void attend_rows(const CUtensorMap &km, const CUtensorMap &vm, const KvAttnArgs &a)
{
    using S = Shape<DT, NT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<DT, NT> &sm = *reinterpret_cast<Smem<DT, NT> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int *before = reinterpret_cast<int *>(&sm + 1);  // units of sequences < b
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < S::kBufs; ++i) mbar_init(&sm.full[w][i], 1);
        sm.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    grid_dep_launch();
    if (!a.behind_tiles) grid_dep_wait();  // queries, cache and batch arrays may come from the kernel before

    // units of every sequence, summed up: each thread takes a run of sequences
    const bool split = a.partials != nullptr;
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    int shift = kUnitShift;
    auto units_of = [&](int b) {
        const int len = a.seq_len[b];
        const KvSpan s = kv_span(a.cu_q[b], a.cu_q[b + 1], len, a.M, a.capacity);
        if (len > a.capacity) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
        if (int64_t(s.n) * a.group > a.few_rows) return int64_t(0);
        return kv_tiles(s.n, a.group, S::kRows) * a.kv_heads * (split ? kTileUnits + kv_units(s.len, 1 << shift) : 1);
    };
    int64_t mine, sum, all;
    for (;; ++shift) {  // (larger units where their count would not fit: more than 2^36 keys)
        mine = 0;
        for (int i = 0; i < per; ++i)
            if (tid * per + i < a.n_seqs) mine += units_of(tid * per + i);
        sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) sm.sums[warp] = sum;
        __syncthreads();
        all = 0;
        int64_t below = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) below += sm.sums[w];
            all += sm.sums[w];
        }
        sum += below - mine;
        if (all <= kMostUnits || shift == 30) break;
        __syncthreads();
    }
    const int total = int(min(all, int64_t(0x7fffffff)));
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < a.n_seqs) {
            before[b] = int(sum);
            sum += per > 1 ? units_of(b) : mine;
        }
    }
    if (tid == 0) before[a.n_seqs] = total;
    __syncthreads();

    // no more shares than units, so that no block between a tile's first and last is without one
    const int least = split ? kTileUnits + kLeastUnits : 1;
    const int grid = min(int(gridDim.x), (total + least - 1) / least), cta = blockIdx.x;
    if (cta >= grid) return;
    int u = share_of(total, cta, grid);
    const int u_end = share_of(total, cta + 1, grid);
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int kSlot = S::kRows * S::kRowFloats;
    // the block's next part of a tile (u: the unit behind it)
    auto next_part = [&](Tile &t) {
        while (u < u_end) {
            int next;
            t = tile_of<S::kRows>(a, before, shift, u, u_end, next);
            u = next;
            if (next > t.u0) return true;  // (else none of the tile's keys)
        }
        return false;
    };
    Walk<DT, NT> walk(a, &km, &vm, sm);
    Tile t, ahead, kept[2];
    bool kept_any[2] = {false, false};  // partials of a tile that began before, of one that ends behind
    bool more = next_part(t);
    if (more) walk.begin(t);
#pragma unroll 1
    while (more) {
        State<DT, NT> st;
        walk.template run<F8, BF16>(st);
        more = next_part(ahead);
        if (more) walk.begin(ahead);
        float *slot = t.whole ? nullptr : a.partials + int64_t(2 * cta + (t.first ? 1 : 0)) * kSlot;
        join<T, DT, NT>(a, sm, t, st, slot);
        if (!t.whole) {
            if (t.first) kept[1] = t;
            else kept[0] = t;
            kept_any[t.first] = true;
        }
        t = ahead;
    }
    // Every partial of the block is written: it arrives at the counters of their tiles (of the
    // tile's first block), and joins the parts of those that it is the last to arrive at.
    if (!kept_any[0] && !kept_any[1]) return;
    if (tid == 0) {
        auto owner = [&](int x) {
            int c = int(unsigned(int64_t(x) * grid / total));  // at or next to the block that holds unit x
            while (c > 0 && share_of(total, c, grid) > x) --c;
            while (share_of(total, c + 1, grid) <= x) ++c;
            return c;
        };
        int c0[2], parts[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (kept_any[i]) {
                c0[i] = i ? cta : owner(kept[i].u0);
                parts[i] = (i ? owner(kept[i].u1 - 1) : (kept[i].u1 - 1 < u_end ? cta : owner(kept[i].u1 - 1))) - c0[i] + 1;
            }
        fence_gpu();  // the block's partials, seen by this thread at the barrier, before its arrivals
        bool last[2] = {false, false};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (kept_any[i]) last[i] = atomicInc(&a.arrivals[c0[i]], unsigned(parts[i] - 1)) == unsigned(parts[i] - 1);
        if (last[0] || last[1]) fence_gpu();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sm.first[i] = last[i] ? c0[i] : 0;
            sm.parts[i] = last[i] ? parts[i] : 0;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (kept_any[i] && sm.parts[i])
            join_parts<T, DT, NT>(a, kept[i], a.partials + int64_t(sm.first[i]) * (2 * kSlot), sm.parts[i]);
}

template <bool F8, bool BF16, int DT, int NT>
__global__ void __launch_bounds__(kThreads, Shape<DT, NT>::kPerSm)
kv_attn_rows_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                    const __grid_constant__ KvAttnArgs a)
{
    attend_rows<F8, BF16, DT, NT>(km, vm, a);
    if (a.behind_tiles) grid_dep_wait();
}

struct RowsPlan {
    const void *fn;
    int per_sm;
    size_t smem;    // without the unit counts
    int row_bytes;  // of a copied box
    int keys;       // of a stage
};

template <bool F8, bool BF16, int DT, int NT>
RowsPlan rows_plan()
{
    using S = Shape<DT, NT>;
    return {reinterpret_cast<const void *>(kv_attn_rows_kernel<F8, BF16, DT, NT>), S::kPerSm,
            sizeof(Smem<DT, NT>) + 1024, S::kRowBytes, S::kKeys};
}

template <bool F8, bool BF16>
RowsPlan rows_plan(int head_dim, bool two)
{
    if (head_dim <= 64) return two ? rows_plan<F8, BF16, 64, 2>() : rows_plan<F8, BF16, 64, 1>();
    if (head_dim <= 128) return two ? rows_plan<F8, BF16, 128, 2>() : rows_plan<F8, BF16, 128, 1>();
    return two ? rows_plan<F8, BF16, 256, 2>() : rows_plan<F8, BF16, 256, 1>();
}

constexpr int kMostPerSm = 2;
constexpr int kFewRows = 16;
// two partial slots a block in the workspace's 64 KB per SM: two blocks of 8 rows of 132 binary32
// values, or one of 16 rows of 260
static_assert(2 * 2 * 8 * (128 + 4) * 4 <= 65536 && 2 * 16 * (256 + 4) * 4 <= 65536, "");

}  // namespace

// Partials of two slots for every block, then the arrival counters (self-resetting).
size_t kv_attn_rows_workspace()
{
    return ws_scratch_bytes() + size_t(device_info().sm_count) * kMostPerSm * sizeof(unsigned);
}

// Keys and values as (page and head, slot, byte): bytes behind the head are not read, the copy
// fills zeros beyond the first dimension.
wq_status encode_cache(CUtensorMap *km, CUtensorMap *vm, const KvAttnArgs &a, int row_bytes, int rows)
{
    const uint64_t dims[3] = {uint64_t(a.head_dim), uint64_t(1) << a.page_shift, uint64_t(a.num_pages) * a.kv_heads};
    const uint64_t strides[2] = {uint64_t(a.pitch), uint64_t(a.pitch) << a.page_shift};
    const uint32_t box[3] = {uint32_t(row_bytes), uint32_t(rows), 1};
    wq_status rc = encode_tmap(km, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.k, dims, strides, box, row_bytes);
    return rc != WQ_OK ? rc : encode_tmap(vm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.v, dims, strides, box, row_bytes);
}

void set_attn_launch(PreparedLaunch &L, const void *fn, unsigned blocks, int threads, size_t smem, const CUtensorMap &km,
                     const CUtensorMap &vm, const KvAttnArgs &a)
{
    static_assert(sizeof(CUtensorMap) == 128 && sizeof(KvAttnArgs) <= 256, "argument layout");
    L.func = fn;
    L.grid = dim3(blocks);
    L.block = dim3(unsigned(threads));
    L.smem = smem;
    memcpy(L.args, &km, sizeof km);
    memcpy(L.args + 128, &vm, sizeof vm);
    memcpy(L.args + 256, &a, sizeof a);
    for (int i = 0; i < 3; ++i) L.argp[i] = L.args + 128 * i;
    L.nargs = 3;
}

wq_status kv_attn_rows(const KvAttnArgs &a, bool bf16, bool f8, cudaStream_t st)
{
    // 16 rows a tile where sequences bring more than 8 rows per key head on average
    const bool two = int64_t(a.M) * a.group > int64_t(8) * a.n_seqs;
    const RowsPlan p = f8 ? (bf16 ? rows_plan<true, true>(a.head_dim, two) : rows_plan<true, false>(a.head_dim, two))
                          : (bf16 ? rows_plan<false, true>(a.head_dim, two) : rows_plan<false, false>(a.head_dim, two));
    const size_t smem = p.smem + size_t(a.n_seqs + 1) * sizeof(int);
    if (cudaFuncSetAttribute(p.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(p.smem + (kKvMaxSeqs + 1) * sizeof(int))) != cudaSuccess)
        return check_launch("cudaFuncSetAttribute(kv_attn_rows_kernel)");
    CUtensorMap km, vm;
    wq_status rc = encode_cache(&km, &vm, a, p.row_bytes, std::min(1 << a.page_shift, p.keys));
    if (rc != WQ_OK) return rc;
    PreparedLaunch L;
    set_attn_launch(L, p.fn, unsigned(device_info().sm_count * p.per_sm), kThreads, smem, km, vm, a);
    return launch_prepared(L, st, "kv_attn_rows_kernel");
}

}  // namespace wq

using namespace wq;

extern "C" size_t kv_attention_workspace_size(int64_t M, int32_t q_heads, const wq_kv_cache *cache,
                                              const wq_kv_batch *batch)
{
    if (check_kv(cache, batch, WQ_F16, M, q_heads) != WQ_OK) return 0;
    return kv_attn_rows_workspace();
}

extern "C" wq_status kv_attention(const void *q, wq_dtype dt, int64_t M, int32_t q_heads, const wq_kv_cache *cache,
                                  const wq_kv_batch *batch, float sm_scale, void *out, void *workspace, size_t ws_bytes,
                                  cudaStream_t stream)
{
    wq_status rc = check_kv(cache, batch, dt, M, q_heads);
    if (rc != WQ_OK) return rc;
    if (!q || !out) return fail(WQ_ERR_INVALID_ARG, "q and out must be non-null");
    if (!std::isfinite(sm_scale)) return fail(WQ_ERR_INVALID_ARG, "sm_scale must be finite");
    if (!aligned16(q) || !aligned16(out) || (workspace && !aligned16(workspace)))
        return fail(WQ_ERR_ALIGNMENT, "q, out and workspace must be 16-byte aligned");
    KvAttnArgs a{};
    a.q = q;
    a.out = out;
    a.k = static_cast<const uint8_t *>(cache->k);
    a.v = static_cast<const uint8_t *>(cache->v);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.cu_q = batch->cu_q;
    a.seq_len = batch->seq_len;
    a.block_table = batch->block_table;
    a.num_pages = cache->num_pages;
    a.n_seqs = int(batch->n_seqs);
    a.max_pages = int(batch->max_pages);
    a.M = int(M);
    a.q_heads = q_heads;
    a.kv_heads = cache->kv_heads;
    a.group = q_heads / cache->kv_heads;
    a.head_dim = cache->head_dim;
    while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
    a.pitch = kv_pitch(cache->head_dim);
    a.capacity = int(batch->max_pages * cache->page_size);
    a.sm_scale = sm_scale;
    if (workspace && ws_bytes >= kv_attn_rows_workspace()) {
        a.partials = static_cast<float *>(workspace);
        a.arrivals = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(workspace) + ws_scratch_bytes());
    }
    // Sequences with up to kFewRows rows per key head are bound by reading their keys once and go
    // to the key-split kernel, the others to the tile kernel (heads up to 128).  One launch
    // where sequences bring that few rows on average, right for any distribution.
    const bool bf16 = dt == WQ_BF16, f8 = cache->format == WQ_FMT_E4M3;
    const bool tiles = a.head_dim <= 128 && M * a.group > kFewRows * batch->n_seqs;
    a.few_rows = tiles ? kFewRows : 0x7fffffff;
    if (tiles) {
        rc = kv_attn_tiles(a, bf16, f8, stream);
        if (rc != WQ_OK) return rc;
        a.behind_tiles = true;
    }
    return kv_attn_rows(a, bf16, f8, stream);
}
