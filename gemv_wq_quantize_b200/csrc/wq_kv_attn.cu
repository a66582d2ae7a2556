// wq_kv_attn.cu -- kv_attention for few rows per key head (decode and draft verification):
// attention over the paged 8-bit cache, split over the whole GPU by key ranges.
//
// Mathematics: for a query row q of position p and the keys j <= p of its sequence,
//   s_j = sm_scale * ks[page(j)] * (q . kc_j),   out = sum_j softmax(s)_j vs[page(j)] vc_j
// with the codes kc, vc exact in binary16, products on mma.sync with binary32 accumulation, one
// pass with a running maximum and sum, and the two page scales applied in binary32.
//
// Bound by reading the cache once: a group of query heads shares a key head's codes, so the
// rows of (sequence, key head) form the 8-wide N side of both products (S^T = K Q^T and
// O^T = V^T P^T): the codes are the 16-row A operand, nothing is wasted on padding up to 8 rows,
// and codes go from global memory straight into the registers of the lane that multiplies them
// (a dot product may take its dimensions in any order, so a lane's 16 contiguous bytes of a key
// are its fragments of four steps; a lane's 16 contiguous bytes of four values are its fragments
// of eight row tiles).  No shared memory on the way, so many loads stay in flight.
//
// Work split: tiles (sequence, key head, 8 * NT rows) are cut into units of kUnit keys, and the
// persistent blocks take equal contiguous shares of all units, whatever the lengths.  A tile cut
// over several blocks leaves partial sums in the workspace; the last block to arrive adds them
// in the order of their keys, so the result does not depend on which block that is.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "wq_act.cuh"
#include "wq_kv_attn.cuh"

namespace wq {

__device__ int g_kv_attn_error;

int kv_attn_read_error()
{
    int v = 0, zero = 0;
    cudaMemcpyFromSymbol(&v, g_kv_attn_error, sizeof v);
    cudaMemcpyToSymbol(g_kv_attn_error, &zero, sizeof zero);
    return v;
}

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 64;  // keys of a unit: the granule of the split

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

__device__ __forceinline__ uint4 ldg_stream(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg_stream8(const uint8_t *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// DT: head_dim rounded up to 64, 128 or 256.  NT: tiles of 8 rows.
template <int DT, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = DT >= 256 || NT > 1 ? 1 : 2;  // 16-key steps of an iteration
    static constexpr int kRowFloats = DT + 2;    // a partial row: sums, maximum, weight sum
};

// A row of sums in shared memory and in the workspace is kept in the order of the fragments:
// place 16 i + 2 g + e holds dimension DT / 8 * g + 2 i + e (lane (g, j) then stores pairs
// without bank conflicts, rows being DT + 4 apart).
template <int DT>
__device__ __forceinline__ int dim_of(int place)
{
    return DT / 8 * (place % 16 / 2) + 2 * (place / 16) + place % 2;
}

template <int DT, int NT>
struct Smem {
    float o[kWarps][8 * NT][DT + 4];
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    int64_t sums[kWarps + 1];
    unsigned last;
    // then the unit counts of all sequences up to each (n_seqs + 1)
};

// The codes of 16 keys in the registers of a warp.
template <int DT>
struct KeyRegs {
    uint4 r[2][DT / 64];  // lane (g, j): keys g and g + 8, bytes 64 c + 16 j
};
template <int DT>
struct ValRegs {
    uint32_t w[4][DT / 32];  // lane (g, j): keys 2j, 2j + 1, 2j + 8, 2j + 9, bytes DT / 8 * g
};

template <int DT>
__device__ __forceinline__ void load_keys(KeyRegs<DT> &k, const uint8_t *base, int pitch, int g, int j)
{
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < DT / 64; ++c) {
            const int d = 64 * c + 16 * j;
            k.r[t][c] = d < pitch ? ldg_stream(base + (g + 8 * t) * pitch + d) : make_uint4(0, 0, 0, 0);
        }
}

template <int DT>
__device__ __forceinline__ void load_vals(ValRegs<DT> &v, const uint8_t *base, int pitch, int g, int j)
{
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint8_t *p = base + (2 * j + (t & 1) + 8 * (t >> 1)) * pitch;
        if constexpr (DT == 64) {
            const int d = 8 * g;
            const uint2 x = d < pitch ? ldg_stream8(p + d) : make_uint2(0, 0);
            v.w[t][0] = x.x;
            v.w[t][1] = x.y;
        } else {
#pragma unroll
            for (int c = 0; c < DT / 128; ++c) {
                const int d = DT / 8 * g + 16 * c;
                const uint4 x = d < pitch ? ldg_stream(p + d) : make_uint4(0, 0, 0, 0);
                v.w[t][4 * c] = x.x;
                v.w[t][4 * c + 1] = x.y;
                v.w[t][4 * c + 2] = x.z;
                v.w[t][4 * c + 3] = x.w;
            }
        }
    }
}

// One warp's running state over its keys: column n of the products is row n of the tile.
template <int DT, int NT>
struct State {
    float o[NT][DT / 16][4];  // lane (g, j): dimensions of tile i: DT/8 g + 2i and + 1; rows 2j, 2j + 1
    float m[NT][2], l[NT][2];
};

// Queries as B fragments (binary16): k-step c * 4 + w holds, for lane (g, j) and row g, the
// dimensions 64 c + 16 j + 4 w .. + 3.  A bfloat16 row is scaled by a power of two so that its
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
                const int d = 64 * c + 16 * j + 4 * w;
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

// Scores of 16 keys: S^T[key][row], lane (g, j) holds keys g and g + 8, rows 2j and 2j + 1.
template <bool F8, int DT, int NT>
__device__ __forceinline__ void scores(const KeyRegs<DT> &k, const uint32_t (&qf)[NT][DT / 16][2], float (&s)[NT][4])
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
    for (int c = 0; c < DT / 64; ++c) {
        const uint32_t *lo = &k.r[0][c].x, *hi = &k.r[1][c].x;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t x = F8 ? lo[w] : lo[w] ^ 0x80808080u, y = F8 ? hi[w] : hi[w] ^ 0x80808080u;
            const uint32_t f[4] = {widen<F8, 0>(x), widen<F8, 0>(y), widen<F8, 1>(x), widen<F8, 1>(y)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(s[n], f, qf[n][4 * c + w][0], qf[n][4 * c + w][1]);
        }
    }
}

// O^T += vs * (V^T P^T) over 16 keys; p: the weights as B fragments.
template <bool F8, int DT, int NT>
__device__ __forceinline__ void add_values(const ValRegs<DT> &v, const uint32_t (&p)[NT][2], float vs, State<DT, NT> &st)
{
#pragma unroll
    for (int i = 0; i < DT / 16; i += 2) {
        // bytes 2i .. 2i + 3 of the lane's chunk of four keys: row tiles i and i + 1
        const uint32_t x0 = v.w[0][i / 2], x1 = v.w[1][i / 2], x2 = v.w[2][i / 2], x3 = v.w[3][i / 2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t a = prmt(x0, x1, e ? 0x7362 : 0x5140), b = prmt(x2, x3, e ? 0x7362 : 0x5140);
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
    int keys;  // keys that the tile's last row sees
};

// The running state over keys [t0, t1) of the tile, 16-key steps taken in turn by the warps.
template <bool F8, bool BF16, int DT, int NT>
__device__ __forceinline__ void walk_keys(const KvAttnArgs &a, const Tile &t, int t0, int t1, State<DT, NT> &st)
{
    using S = Shape<DT, NT>;
    constexpr int kSpan = 16 * S::kSteps;  // keys of a warp's iteration
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, j = lane % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        st.m[n][0] = st.m[n][1] = -INFINITY;
        st.l[n][0] = st.l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < DT / 16; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) st.o[n][i][x] = 0.f;
    }
    uint32_t qf[NT][DT / 16][2];
    float qs[NT][2];
    load_queries<BF16, DT, NT>(a, t.s, t.head, t.row0, t.rows, g, j, qf, qs);
    int seen[NT][2];  // keys that rows 2j and 2j + 1 see
    int least = t1;   // keys that every row of the tile sees
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = 8 * n + 2 * j + x;
            seen[n][x] = r < t.rows ? t.s.len - t.s.n + (t.row0 + r) / a.group + 1 : 0;
            qs[n][x] *= a.sm_scale * kLog2e;
        }
    least = min(least, t.s.len - t.s.n + t.row0 / a.group + 1);
    const int32_t *table = a.block_table + int64_t(t.b) * a.max_pages;
    const int last_page = (t1 - 1) >> a.page_shift;

    KeyRegs<DT> kr[S::kSteps];
    ValRegs<DT> vr[S::kSteps];
    float ks[S::kSteps], vs[S::kSteps];
    int64_t at[S::kSteps];  // byte offset of the step's codes (page 0 for a bad entry)
    bool ok[S::kSteps];
    auto page_of = [&](int key) { return table[min(key >> a.page_shift, last_page)]; };
    auto place = [&](int i, int entry, int key) {
        const int64_t page = kv_page_ok(entry, a.num_pages);
        ok[i] = page >= 0;
        if (!ok[i] && key < t1) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
        const int64_t p = ok[i] ? page : 0;
        at[i] = kv_code_offset(p, t.head, key & ((1 << a.page_shift) - 1), a.kv_heads, a.page_shift, a.pitch);
        const int64_t si = kv_scale_index(p, t.head, a.kv_heads);
        ks[i] = __ldg(a.k_scale + si);
        vs[i] = ok[i] ? __ldg(a.v_scale + si) : 0.f;
    };
    int key = t0 + warp * kSpan;
    if (key >= t1) return;
    int entry[S::kSteps];
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) entry[i] = page_of(key + 16 * i);
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) {
        place(i, entry[i], key + 16 * i);
        load_keys<DT>(kr[i], a.k + at[i], a.pitch, g, j);
    }
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) load_vals<DT>(vr[i], a.v + at[i], a.pitch, g, j);
    constexpr int kStride = kWarps * kSpan;
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) entry[i] = page_of(key + kStride + 16 * i);

    for (; key < t1; key += kStride) {
        float s[S::kSteps][NT][4];
        float vcur[S::kSteps];
        const bool more = key + kStride < t1;
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
            if (F8 && a.head_dim < a.pitch) {  // bytes behind the head hold anything, NaN codes among it
#pragma unroll
                for (int c = 0; c < DT / 64; ++c)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        if (64 * c + 16 * j + 4 * w >= a.head_dim) (&kr[i].r[0][c].x)[w] = (&kr[i].r[1][c].x)[w] = 0u;
            }
            scores<F8, DT, NT>(kr[i], qf, s[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[i][n][x] *= ks[i] * qs[n][x & 1];
            const int first = key + 16 * i;
            if (first + 16 > least || !ok[i]) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int k = first + g + 8 * (x >> 1);
                        if (k >= min(seen[n][x & 1], t1) || !ok[i]) s[i][n][x] = -INFINITY;
                    }
                // slots behind the last key hold anything, e4m3 NaN codes among it
                if (F8 && first + 16 > t1) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (first + 2 * j + (c & 1) + 8 * (c >> 1) >= t1)
#pragma unroll
                            for (int w = 0; w < DT / 32; ++w) vr[i].w[c][w] = 0u;
                }
            }
            vcur[i] = vs[i];
        }
        // the next keys are on their way while the softmax and the values are worked on
        if (more) {
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
                place(i, entry[i], key + kStride + 16 * i);
                load_keys<DT>(kr[i], a.k + at[i], a.pitch, g, j);
                entry[i] = page_of(key + 2 * kStride + 16 * i);
            }
        }
        uint32_t p[S::kSteps][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mx[2] = {st.m[n][0], st.m[n][1]};
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) mx[x & 1] = fmaxf(mx[x & 1], s[i][n][x]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
            }
            if (__any_sync(0xffffffffu, mx[0] > st.m[n][0] || mx[1] > st.m[n][1])) {
                // -inf - -inf: no key seen yet, nothing to rescale
                const float f0 = mx[0] == st.m[n][0] ? 1.f : exp2_approx(st.m[n][0] - mx[0]);
                const float f1 = mx[1] == st.m[n][1] ? 1.f : exp2_approx(st.m[n][1] - mx[1]);
                st.l[n][0] *= f0;
                st.l[n][1] *= f1;
#pragma unroll
                for (int i = 0; i < DT / 16; ++i) {
                    st.o[n][i][0] *= f0;
                    st.o[n][i][1] *= f1;
                    st.o[n][i][2] *= f0;
                    st.o[n][i][3] *= f1;
                }
                st.m[n][0] = mx[0];
                st.m[n][1] = mx[1];
            }
            const float base[2] = {mx[0] == -INFINITY ? 0.f : mx[0] - kRaise, mx[1] == -INFINITY ? 0.f : mx[1] - kRaise};
#pragma unroll
            for (int i = 0; i < S::kSteps; ++i) {
                float w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    w[x] = exp2_approx(s[i][n][x] - base[x & 1]);
                    st.l[n][x & 1] += w[x];
                }
                // weights to binary16: half a step is 2^-12 of each, of either sign
                p[i][n][0] = trans8x8(act_t2<__half>(w[0], w[1]));
                p[i][n][1] = trans8x8(act_t2<__half>(w[2], w[3]));
            }
        }
#pragma unroll
        for (int i = 0; i < S::kSteps; ++i) {
            add_values<F8, DT, NT>(vr[i], p[i], vcur[i], st);
            if (more) load_vals<DT>(vr[i], a.v + at[i], a.pitch, g, j);
        }
    }
}

template <bool F8, bool BF16, int DT, int NT>
__global__ void __launch_bounds__(kThreads, DT >= 256 || NT > 1 ? 2 : 3)
kv_attn_rows_kernel(const __grid_constant__ KvAttnArgs a)
{
    using S = Shape<DT, NT>;
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<DT, NT> &sm = *reinterpret_cast<Smem<DT, NT> *>(smem_raw);
    int64_t *before = reinterpret_cast<int64_t *>(smem_raw + sizeof(Smem<DT, NT>));  // units of sequences < b
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    grid_dep_launch();
    grid_dep_wait();  // queries, cache and batch arrays may come from the kernel before

    // units of every sequence, summed up: each thread takes a run of sequences
    const bool split = a.partials != nullptr;
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    auto units_of = [&](int b) {
        const int len = a.seq_len[b];
        const KvSpan s = kv_span(a.cu_q[b], a.cu_q[b + 1], len, a.M, a.capacity);
        if (len > a.capacity) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
        if (int64_t(s.n) * a.group > a.few_rows) return int64_t(0);
        return kv_tiles(s.n, a.group, S::kRows) * (split ? kv_units(s.len, kUnit) : 1) * a.kv_heads;
    };
    int64_t mine = 0;
    for (int i = 0; i < per; ++i)
        if (tid * per + i < a.n_seqs) mine += units_of(tid * per + i);
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) sm.sums[warp] = sum;
    __syncthreads();
    int64_t run = sum - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) run += sm.sums[w];
        total += sm.sums[w];
    }
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < a.n_seqs) {
            before[b] = run;
            run += per > 1 ? units_of(b) : mine;
        }
    }
    if (tid == 0) before[a.n_seqs] = total;
    __syncthreads();

    // no more shares than units, so that no block between a tile's first and last is without one
    const int grid = int(min(int64_t(gridDim.x), total)), cta = blockIdx.x;
    if (cta >= grid) return;
    int64_t u = kv_share(total, cta, grid);
    const int64_t u_end = kv_share(total, cta + 1, grid);
    while (u < u_end) {
        // the sequence of unit u: the last b with before[b] <= u (empty ones have no units)
        int lo = 0, hi = a.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (before[mid] <= u) lo = mid;
            else hi = mid;
        }
        Tile t;
        t.b = lo;
        t.s = kv_span(a.cu_q[lo], a.cu_q[lo + 1], a.seq_len[lo], a.M, a.capacity);
        const int64_t units = split ? kv_units(t.s.len, kUnit) : 1;
        const int64_t tiles = kv_tiles(t.s.n, a.group, S::kRows);
        const int64_t item = (u - before[lo]) / units;  // (key head, tile) of the sequence
        const int64_t item_u0 = before[lo] + item * units;
        t.head = int(item / tiles);
        t.row0 = int(item % tiles) * S::kRows;
        t.rows = min(S::kRows, t.s.n * a.group - t.row0);
        t.keys = max(0, t.s.len - t.s.n + (t.row0 + t.rows - 1) / a.group + 1);
        const int64_t item_end = item_u0 + units, seg_end = min(item_end, u_end);
        // keys of this block's units of the tile
        const int t0 = split ? int(min(int64_t(t.keys), (u - item_u0) * kUnit)) : 0;
        const int t1 = split ? int(min(int64_t(t.keys), (seg_end - item_u0) * kUnit)) : t.keys;
        const bool whole = u == item_u0 && seg_end == item_end;

        State<DT, NT> st;
        walk_keys<F8, BF16, DT, NT>(a, t, t0, t1, st);

        // the warps' states, joined in shared memory
        const int g = lane / 4, j = lane % 4;
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
#pragma unroll
            for (int i = 0; i < DT / 16; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    *reinterpret_cast<float2 *>(&sm.o[warp][8 * n + 2 * j + x][16 * i + 2 * g]) =
                        make_float2(st.o[n][i][x], st.o[n][i][2 + x]);
        }
        __syncthreads();
        // partial of this block, or the finished rows
        float *slot = nullptr;
        if (!whole) slot = a.partials + int64_t(2 * cta + (u == item_u0 ? 1 : 0)) * S::kRows * S::kRowFloats;
        for (int e = tid; e < S::kRows * (DT / 2); e += kThreads) {
            const int r = e / (DT / 2), at = 2 * (e % (DT / 2)), d = dim_of<DT>(at);
            float m = sm.m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sm.m[w][r]);
            float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = sm.m[w][r];
                const float f = mw == -INFINITY ? 0.f : exp2_approx(mw - m);
                l += f * sm.l[w][r];
                x += f * sm.o[w][r][at];
                y += f * sm.o[w][r][at + 1];
            }
            if (whole) {
                if (r < t.rows && d < a.head_dim) {
                    const int row = t.row0 + r;
                    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
                    uint16_t *o = static_cast<uint16_t *>(a.out) +
                                  (int64_t(t.s.q0 + row / a.group) * a.q_heads + t.head * a.group + row % a.group) *
                                      a.head_dim + d;
                    *reinterpret_cast<uint32_t *>(o) = act_t2<T>(x * inv, y * inv);
                }
            } else {
                *reinterpret_cast<float2 *>(slot + r * S::kRowFloats + at) = make_float2(x, y);
                if (at == 0) *reinterpret_cast<float2 *>(slot + r * S::kRowFloats + DT) = make_float2(m, l);
            }
        }
        if (!whole) {
            // the blocks of a tile arrive at the counter of the tile's first block
            const int c0 = [&] {
                int x = int(item_u0 * grid / total);  // near the block that holds unit item_u0
                while (x > 0 && kv_share(total, x, grid) > item_u0) --x;
                while (kv_share(total, x + 1, grid) <= item_u0) ++x;
                return x;
            }();
            const int c1 = [&] {
                int x = int((item_end - 1) * grid / total);
                while (x > 0 && kv_share(total, x, grid) > item_end - 1) --x;
                while (kv_share(total, x + 1, grid) <= item_end - 1) ++x;
                return x;
            }();
            __threadfence();
            __syncthreads();
            if (tid == 0) sm.last = atomicInc(&a.arrivals[c0], unsigned(c1 - c0)) == unsigned(c1 - c0);
            __syncthreads();
            if (sm.last) {
                __threadfence();
                const int64_t stride = int64_t(2) * S::kRows * S::kRowFloats;
                const float *p0 = a.partials + int64_t(c0) * stride;  // its second slot, the others' first
                auto part = [&](int c) { return p0 + (c - c0) * stride + (c == c0 ? S::kRows * S::kRowFloats : 0); };
                for (int e = tid; e < t.rows * (DT / 2); e += kThreads) {
                    const int r = e / (DT / 2), at = 2 * (e % (DT / 2)), d = dim_of<DT>(at);
                    if (d >= a.head_dim) continue;
                    float m = -INFINITY;
                    for (int c = c0; c <= c1; ++c) m = fmaxf(m, __ldcg(part(c) + r * S::kRowFloats + DT));
                    float l = 0.f, x = 0.f, y = 0.f;
                    for (int c = c0; c <= c1; ++c) {
                        const float *row = part(c) + r * S::kRowFloats;
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(row + DT));
                        const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
                        const float2 xy = __ldcg(reinterpret_cast<const float2 *>(row + at));
                        l += f * ml.y;
                        x += f * xy.x;
                        y += f * xy.y;
                    }
                    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
                    const int row = t.row0 + r;
                    uint16_t *out = static_cast<uint16_t *>(a.out) +
                                    (int64_t(t.s.q0 + row / a.group) * a.q_heads + t.head * a.group + row % a.group) *
                                        a.head_dim + d;
                    *reinterpret_cast<uint32_t *>(out) = act_t2<T>(x * inv, y * inv);
                }
            }
        }
        __syncthreads();  // shared memory is reused by the next tile
        u = seg_end;
    }
}

struct RowsPlan {
    const void *fn;
    int per_sm;      // resident blocks
    size_t smem;     // without the unit counts
};

template <bool F8, bool BF16, int DT>
RowsPlan rows_plan(bool two)
{
    if (two)
        return {reinterpret_cast<const void *>(kv_attn_rows_kernel<F8, BF16, DT, 2>), 2, sizeof(Smem<DT, 2>)};
    return {reinterpret_cast<const void *>(kv_attn_rows_kernel<F8, BF16, DT, 1>), DT >= 256 ? 2 : 3, sizeof(Smem<DT, 1>)};
}

template <bool F8, bool BF16>
RowsPlan rows_plan(int head_dim, bool two)
{
    if (head_dim <= 64) return rows_plan<F8, BF16, 64>(two);
    if (head_dim <= 128) return rows_plan<F8, BF16, 128>(two);
    return rows_plan<F8, BF16, 256>(two);
}

constexpr int kMostPerSm = 3;
constexpr int kFewRows = 16;
// two partial slots a block: the largest of 3 blocks of 8 rows of 130 binary32 values, 2 blocks
// of 16 rows of 258
static_assert(3 * 2 * 8 * (128 + 2) * 4 <= 65536 && 2 * 2 * 16 * (256 + 2) * 4 <= 2 * 65536, "");

}  // namespace

// Partials of two slots for every block, then the arrival counters (self-resetting).
static size_t rows_partial_bytes() { return size_t(device_info().sm_count) * 2 * 2 * 16 * (256 + 2) * 4; }

size_t kv_attn_rows_workspace()
{
    return std::max(rows_partial_bytes(), ws_scratch_bytes()) + size_t(device_info().sm_count) * kMostPerSm * sizeof(unsigned);
}

wq_status kv_attn_rows(const KvAttnArgs &a, bool bf16, bool f8, cudaStream_t st)
{
    // 16 rows a tile where sequences bring more than 8 rows per key head on average
    const bool two = int64_t(a.M) * a.group > int64_t(8) * a.n_seqs;
    const RowsPlan p = f8 ? (bf16 ? rows_plan<true, true>(a.head_dim, two) : rows_plan<true, false>(a.head_dim, two))
                          : (bf16 ? rows_plan<false, true>(a.head_dim, two) : rows_plan<false, false>(a.head_dim, two));
    const size_t smem = p.smem + size_t(a.n_seqs + 1) * sizeof(int64_t);
    if (cudaFuncSetAttribute(p.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(p.smem + (kKvMaxSeqs + 1) * 8)) != cudaSuccess)
        return check_launch("cudaFuncSetAttribute(kv_attn_rows_kernel)");
    PreparedLaunch L;
    L.set(p.fn, dim3(unsigned(device_info().sm_count * p.per_sm)), dim3(kThreads), smem, a);
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
    const size_t need = kv_attn_rows_workspace();
    if (workspace && ws_bytes >= need) {
        a.partials = static_cast<float *>(workspace);
        a.arrivals = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(workspace) +
                                                  std::max(rows_partial_bytes(), ws_scratch_bytes()));
    }
    // Sequences with up to kFewRows rows per key head are bound by reading their keys once and go
    // to the key-split kernel, the others to the tile kernel (heads up to 128).  One launch
    // where sequences bring that few rows on average, right for any distribution.
    const bool bf16 = dt == WQ_BF16, f8 = cache->format == WQ_FMT_E4M3;
    const bool tiles = a.head_dim <= 128 && M * a.group > kFewRows * batch->n_seqs;
    a.few_rows = tiles ? kFewRows : 0x7fffffff;
    rc = kv_attn_rows(a, bf16, f8, stream);
    return rc == WQ_OK && tiles ? kv_attn_tiles(a, bf16, f8, stream) : rc;
}
