// wq_kv_append.cu -- kv_append: rotary positions on the queries and keys of a fused QKV row,
// and the append of keys and values to a paged 8-bit cache, in one launch for sm_100a.
//
// Mathematics: a rotated pair is (a c - b s, b c + a s), every product and sum one binary32
// rounding; a page and head has one scale, max(scale before, max|x| * binary32(1 / qmax)) over the call's new
// tokens x of the page, and codes of x / scale.  A scale that grows re-codes the page's earlier
// tokens by (scale before / scale).
//
// Work items.  The maximum over a page's new tokens needs one owner per (page, head): a block
// owns one (sequence, page) item and a head's keys or values; which sequence an item belongs to
// follows from cu_q alone (wq_kv.h), found by all threads of the block looking at once.  For a
// sequence of few tokens a block owns the sequence and four heads, a warp for each's keys or
// values.  A group of WPT
// warps owns the keys or the values of one head: every lane holds four neighbouring values of a
// row (so the partner of a rotated value is one more 8-byte load of the same row, not a
// shuffle), the rows of the page go over the group's warps, and the rotated values stay in
// registers between the maximum and the codes.  Other blocks of the same launch turn the
// queries.
//
// Bound by instruction issue for long runs (rotation, codes), else by the launch and the chain of
// table, row, maximum and codes.  Measured (device time, calls back to back in a graph), 32 query heads:
// 8192 tokens in six runs, 8 key heads of 128: 37 us, 3.2 TB/s (108 us with branches around the loads and a
// division a code); 48 sequences of 1 to 6 tokens, 32 key heads of 100: 8.0 us; 16 of one token, 32 key
// heads of 128: 3.5 us.  These repeat a call, so no page's scale grows.  Where it does, a warp re-codes the
// page's earlier rows one after the other: 16 single tokens, filling pages of 16 from their start with
// ever larger values, take 6.7 us a step, pages of 64 16.6.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cfloat>

#include "wq_act.cuh"
#include "wq_host.h"
#include "wq_kv.h"

namespace wq {

__device__ int g_kv_append_error;

int kv_append_read_error()
{
    int v = 0, zero = 0;
    cudaMemcpyFromSymbol(&v, g_kv_append_error, sizeof v);
    cudaMemcpyToSymbol(g_kv_append_error, &zero, sizeof zero);
    return v;
}

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeldFloats = 32;  // binary32 values of a page that a lane keeps in registers

// How the values of a row turn: kPairs: partners among a lane's four values, cos / sin in aligned
// pairs; kHalf: partners rope_dim / 2 away, everything 8-byte aligned (rope_dim a multiple of 8);
// kHalf2: the same with 4-byte alignment (a multiple of 4); kAny: the rest; kNone.
enum Mode { kNone, kPairs, kHalf, kHalf2, kAny };

struct AppendArgs {
    const void *qkv;
    void *q_out;
    const float *rope;
    wq_kv_cache c;
    const int32_t *cu_q, *seq_len, *block_table;
    int n_seqs, max_pages, M, q_heads;
    int rope_dim;
    int page_shift, pitch;
    int limit;          // positions below it have a place: those of the block table's row and of the rope table
    bool pairs;         // WQ_ROPE_PAIRS
    int items;          // (sequence, page) items of long runs
    int run_blocks;     // and the blocks that take them
    int parts;          // blocks of a sequence of few tokens
    int q_tokens;       // tokens of a query block
};

// Four neighbouring values d .. d + 3 of a head row and their rotation.  Loads and arithmetic are
// apart, and the loads of a row that does not turn (or of a lane behind the head) go to a valid
// address and are not used: without branches around them the loads of many rows are in flight
// before the first is worked on.  Rows, batch arrays and scales are read with plain loads: the kernel
// ahead may write them while this one is already resident, which the read-only path does not allow.
// (The rope table is no such kernel's output.)
struct Turn {
    float c[4], s[4];
};
struct Raw {
    uint2 x, p;  // the values and (but for kPairs) their partners
};

template <Mode MODE>
__device__ __forceinline__ Turn load_turn(const AppendArgs &a, const float *tab, int d)
{
    Turn t{};
    const int half = a.rope_dim / 2;
    if constexpr (MODE == kPairs) {
        const int u = d < a.rope_dim ? d / 2 : 0;
        const float2 c = __ldg(reinterpret_cast<const float2 *>(tab + u));
        const float2 s = __ldg(reinterpret_cast<const float2 *>(tab + half + u));
        t.c[0] = t.c[1] = c.x;
        t.c[2] = t.c[3] = c.y;
        t.s[0] = t.s[1] = s.x;
        t.s[2] = t.s[3] = s.y;
    } else if constexpr (MODE == kHalf) {
        const int u = d < half ? d : (d < a.rope_dim ? d - half : 0);
        const float4 c = __ldg(reinterpret_cast<const float4 *>(tab + u));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(tab + half + u));
        t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
        t.s[0] = s.x; t.s[1] = s.y; t.s[2] = s.z; t.s[3] = s.w;
    } else if constexpr (MODE == kHalf2) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const int e = min(d + i, a.rope_dim - 2), u = e < half ? e : e - half;
            const float2 c = __ldg(reinterpret_cast<const float2 *>(tab + u));
            const float2 s = __ldg(reinterpret_cast<const float2 *>(tab + half + u));
            t.c[i] = c.x;
            t.c[i + 1] = c.y;
            t.s[i] = s.x;
            t.s[i + 1] = s.y;
        }
    } else if constexpr (MODE == kAny) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = min(d + i, a.rope_dim - 1);
            const int u = a.pairs ? e / 2 : (e < half ? e : e - half);
            t.c[i] = __ldg(tab + u);
            t.s[i] = __ldg(tab + half + u);
        }
    }
    return t;
}

template <typename T, Mode MODE>
__device__ __forceinline__ Raw load_raw(const AppendArgs &a, const T *row, int d)
{
    Raw r;
    r.x = *reinterpret_cast<const uint2 *>(row + d);
    if constexpr (MODE == kHalf) {
        const int half = a.rope_dim / 2;
        r.p = *reinterpret_cast<const uint2 *>(row + (d < half ? d + half : (d < a.rope_dim ? d - half : d)));
    } else if constexpr (MODE == kHalf2) {
        const int half = a.rope_dim / 2;
        uint32_t p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = min(d + 2 * i, a.rope_dim - 2);
            p[i] = *reinterpret_cast<const uint32_t *>(row + (e < half ? e + half : e - half));
        }
        r.p = make_uint2(p[0], p[1]);
    } else if constexpr (MODE == kAny) {
        const uint16_t *w = reinterpret_cast<const uint16_t *>(row);
        const int half = a.rope_dim / 2;
        uint16_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = min(d + i, a.rope_dim - 1);
            p[i] = w[a.pairs ? (e ^ 1) : (e < half ? e + half : e - half)];
        }
        r.p = make_uint2(p[0] | uint32_t(p[1]) << 16, p[2] | uint32_t(p[3]) << 16);
    }
    return r;
}

// A value x with partner p turns to x c - p s (first of its pair) or x c + p s (second).
template <typename T, Mode MODE>
__device__ __forceinline__ void turn4(const AppendArgs &a, int d, const Raw &r, const Turn &t, float (&y)[4])
{
    const float2 lo = act_f2<T>(r.x.x), hi = act_f2<T>(r.x.y);
    const float x[4] = {lo.x, lo.y, hi.x, hi.y};
    float p[4] = {x[1], x[0], x[3], x[2]};
    if constexpr (MODE == kHalf || MODE == kHalf2 || MODE == kAny) {
        const float2 plo = act_f2<T>(r.p.x), phi = act_f2<T>(r.p.y);
        p[0] = plo.x; p[1] = plo.y; p[2] = phi.x; p[3] = phi.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (MODE == kNone) {
            y[i] = x[i];
        } else {
            const int e = d + i;
            const bool first = MODE == kPairs || (MODE == kAny && a.pairs) ? !(i & 1) : e < a.rope_dim / 2;
            const float xc = __fmul_rn(x[i], t.c[i]), ps = __fmul_rn(p[i], t.s[i]);
            y[i] = e >= a.rope_dim ? x[i] : (first ? __fsub_rn(xc, ps) : __fadd_rn(xc, ps));
        }
    }
}

// The largest finite magnitude; NaN is stored as 0.  An infinity stays one for the moment (`inf`):
// it saturates once the scale is known.
__device__ __forceinline__ float absmax_finite(float (&y)[4], float m, bool &inf)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (y[i] != y[i]) y[i] = 0.f;
        const float v = fabsf(y[i]);
        inf |= v > FLT_MAX;
        m = v <= FLT_MAX ? fmaxf(m, v) : m;
    }
    return m;
}

template <bool F8>
__device__ __forceinline__ uint32_t store_codes(float (&y)[4], const CodeScale &cs, bool inf)
{
    if (inf) {
        const float most = (F8 ? 448.f : 127.f) * cs.s;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fminf(fmaxf(y[i], -most), most);
    }
    return codes4<F8>(y, cs);
}

// Keys or values of one head of a page, by WPT warps (wi: the warp among them).  CH: chunks of 128
// values of a head (a lane has four of each).  s_max: one value per warp.
template <typename T, bool F8, int WPT, int CH, Mode MODE>
__device__ __forceinline__ void append_rows(const AppendArgs &a, const T *src, const float *tab, const KvPageSpan &ps,
                                            int count, bool live, float *scale, uint8_t *codes, int wi,
                                            float *s_max)
{
    constexpr int kHeld = kHeldFloats / (4 * CH);
    // Rows whose loads are in flight together.  A warp that has a page to itself mostly holds one or
    // two rows: more at once is code to step over (few tokens: 9.6 us with 4, 7.7 with 1).  A row that
    // turns by halves has two loads and a table of its own a lane: more than 2 spill (4096 tokens 36.8
    // us, with 8 40.3; turned by pairs 39.5 and 37.8).
    constexpr int kMost = WPT == 1 ? 1 : MODE == kPairs || MODE == kNone ? 8 : 2, kBatch = kHeld < kMost ? kHeld : kMost;
    const int lane = threadIdx.x % 32, D = a.c.head_dim;
    const int64_t row_stride = int64_t(a.q_heads + 2 * a.c.kv_heads) * D;
    auto dim = [&](int c) { return 4 * (lane + 32 * c); };
    auto at = [&](int c) { return min(dim(c), D - 4); };
    auto turned = [&](int r, int c, float (&y)[4]) {
        turn4<T, MODE>(a, at(c), load_raw<T, MODE>(a, src + r * row_stride, at(c)),
                       load_turn<MODE>(a, tab + int64_t(r) * a.rope_dim, at(c)), y);
    };
    float held[kHeld][CH][4];
    float amax = 0.f, before = 0.f;
    bool inf = false;
    if (live && wi < count) {
        if (ps.off > 0) before = *scale;
#pragma unroll
        for (int i0 = 0; i0 < kHeld; i0 += kBatch) {
            if (wi + i0 * WPT >= count) break;
            Raw raw[kBatch][CH];
            Turn turn[kBatch][CH];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = min(wi + (i0 + i) * WPT, count - 1);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    raw[i][c] = load_raw<T, MODE>(a, src + r * row_stride, at(c));
                    turn[i][c] = load_turn<MODE>(a, tab + int64_t(r) * a.rope_dim, at(c));
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    // a row or lane of the repeated address repeats its values: the maximum is the same
                    turn4<T, MODE>(a, at(c), raw[i][c], turn[i][c], held[i0 + i][c]);
                    amax = absmax_finite(held[i0 + i][c], amax, inf);
                }
        }
        for (int r = wi + kHeld * WPT; r < count; r += WPT)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float y[4];
                turned(r, c, y);
                amax = absmax_finite(y, amax, inf);
            }
        amax = __uint_as_float(warp_umax(__float_as_uint(amax)));
    }
    if constexpr (WPT > 1) {
        if (lane == 0) s_max[wi] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPT; ++i) amax = fmaxf(amax, s_max[i]);
        if (live && wi >= count && ps.off > 0) before = *scale;
        __syncthreads();  // every warp has read the scale before it is replaced
    } else {
        __syncwarp();
    }
    if (!live) return;
    const float now = fmaxf(before, __fmul_rn(amax, kInvQmax<F8>));
    if (wi == 0 && lane == 0) *scale = now;
    if (now > before && ps.off > 0) {  // the page's earlier tokens in the new scale
        const float ratio = __fdiv_rn(before, now);
        const CodeScale one = code_scale(1.f);
        for (int r = wi; r < ps.off; r += WPT)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (dim(c) >= D) continue;
                uint32_t *p = reinterpret_cast<uint32_t *>(codes + int64_t(r) * a.pitch + dim(c));
                const uint32_t w = *p;
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(code_value<F8>(w, i), ratio);
                *p = codes4<F8>(y, one);
            }
    }
    const CodeScale cs = code_scale(now);
    codes += int64_t(ps.off) * a.pitch;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int r = wi + i * WPT;
        if (r >= count) break;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t w = store_codes<F8>(held[i][c], cs, inf);
            if (dim(c) < D) *reinterpret_cast<uint32_t *>(codes + int64_t(r) * a.pitch + dim(c)) = w;
        }
    }
    for (int r = wi + kHeld * WPT; r < count; r += WPT)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float y[4];
            turned(r, c, y);
            absmax_finite(y, 0.f, inf);
            const uint32_t w = store_codes<F8>(y, cs, inf);
            if (dim(c) < D) *reinterpret_cast<uint32_t *>(codes + int64_t(r) * a.pitch + dim(c)) = w;
        }
}

// Keys and values of one page of a sequence.
template <typename T, bool F8, int WPT, int CH, Mode MODE>
__device__ __forceinline__ void append_page(const AppendArgs &a, int b, const KvPageSpan &ps, int part, float *s_max)
{
    constexpr int kTasks = kWarps / WPT;  // (head, keys or values) pairs of the block
    const int tid = threadIdx.x, warp = tid / 32;
    const int pos0 = (ps.page << a.page_shift) + ps.off;
    const int count = kv_placed(ps, a.page_shift, a.limit);
    const int64_t page =
        count > 0 ? kv_page_ok(a.block_table[int64_t(b) * a.max_pages + ps.page], a.c.num_pages) : -1;
    if (tid == 0 && (page < 0 || count < ps.count)) atomicCAS(&g_kv_append_error, kErrNone, kErrRange);
    if (page < 0) return;

    const int task = warp / WPT, wi = warp % WPT;
    const int pair = part * kTasks + task;  // keys of head h, then its values
    const int head = min(pair / 2, a.c.kv_heads - 1), D = a.c.head_dim;
    const bool is_k = (pair & 1) == 0, live = pair < 2 * a.c.kv_heads;
    const T *src = static_cast<const T *>(a.qkv) + int64_t(ps.token) * (a.q_heads + 2 * a.c.kv_heads) * D +
                   int64_t(a.q_heads + (is_k ? 0 : a.c.kv_heads) + head) * D;
    float *scale = (is_k ? a.c.k_scale : a.c.v_scale) + kv_scale_index(page, head, a.c.kv_heads);
    uint8_t *codes = static_cast<uint8_t *>(is_k ? a.c.k : a.c.v) +
                     kv_code_offset(page, head, 0, a.c.kv_heads, a.page_shift, a.pitch);
    if (MODE != kNone && is_k)  // (one answer for the warps of a task, and with WPT > 1 for the block)
        append_rows<T, F8, WPT, CH, MODE>(a, src, a.rope + int64_t(pos0) * a.rope_dim, ps, count, live, scale, codes, wi, s_max);
    else
        append_rows<T, F8, WPT, CH, kNone>(a, src, nullptr, ps, count, live, scale, codes, wi, s_max);
}

// All pages of a sequence of few tokens, a warp for the keys or the values of a head.
template <typename T, bool F8, int CH, Mode MODE>
__device__ __forceinline__ void append_few(const AppendArgs &a, int b, int part)
{
    const KvSpan span = kv_append_span(a.cu_q[b], a.cu_q[b + 1], a.seq_len[b], a.M);
    if (span.n > kKvFewTokens) return;
#pragma unroll 1
    for (int k = 0;; ++k) {
        const KvPageSpan ps = kv_page_span(span, k, a.page_shift);
        if (ps.count == 0) break;
        append_page<T, F8, 1, CH, MODE>(a, b, ps, part, nullptr);
    }
}

// A (sequence, page) item of a long run, all warps for the keys or the values of a head.  False: the
// call has no long run.
template <typename T, bool F8, int CH, Mode MODE, bool RUNS>
__device__ __forceinline__ bool append_item(const AppendArgs &a, int item, int part)
{
    __shared__ float s_max[kWarps];
    __shared__ int s_seq[4];
    const int tid = threadIdx.x;
    if (tid == 0) s_seq[0] = -1;
    __syncthreads();
    bool any = false;
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
        const int q0 = kv_clamp(lo, 0, a.M), q1 = kv_clamp(hi, q0, a.M);
        if (q1 - q0 <= kKvFewTokens) continue;
        any = true;
        if (kv_item_start(q0, b, a.page_shift, RUNS) <= item && item < kv_item_start(q1, b + 1, a.page_shift, RUNS)) {
            s_seq[0] = b;
            s_seq[1] = lo;
            s_seq[2] = hi;
            s_seq[3] = a.seq_len[b];
        }
    }
    if (!__syncthreads_or(any)) return false;
    const int b = s_seq[0];
    if (b >= 0) {
        const KvSpan span = kv_append_span(s_seq[1], s_seq[2], s_seq[3], a.M);
        const KvPageSpan ps = kv_page_span(span, item - kv_item_start(span.q0, b, a.page_shift, RUNS), a.page_shift);
        if (ps.count) append_page<T, F8, kWarps, CH, MODE>(a, b, ps, part, s_max);
    }
    return true;
}

// The queries of q_tokens tokens: kWarps / q_tokens warps take a token's heads in turn.
template <typename T, int CH, Mode MODE>
__device__ __forceinline__ void turn_queries(const AppendArgs &a, int64_t block)
{
    __shared__ int s_pos[kWarps];  // position; -1: no place; -2: not part of a sequence
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t m0 = block * a.q_tokens;
    if (tid < kWarps) s_pos[tid] = -2;
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const KvSpan s = kv_append_span(a.cu_q[b], a.cu_q[b + 1], a.seq_len[b], a.M);
        for (int64_t m = max(int64_t(s.q0), m0); m < min(int64_t(s.q0) + s.n, m0 + a.q_tokens); ++m) {
            const int p = s.len - s.n + int(m - s.q0);
            s_pos[m - m0] = p < 0 || p >= a.limit ? -1 : p;
            if (p >= a.limit) atomicCAS(&g_kv_append_error, kErrNone, kErrRange);
        }
    }
    __syncthreads();
    const int per = kWarps / a.q_tokens, t = warp / per;
    const int64_t m = m0 + t;
    const int pos = s_pos[t];
    if (pos == -2) return;
    const int D = a.c.head_dim;
    const T *src = static_cast<const T *>(a.qkv) + m * int64_t(a.q_heads + 2 * a.c.kv_heads) * D;
    T *dst = static_cast<T *>(a.q_out) + m * int64_t(a.q_heads) * D;
    const float *tab = MODE == kNone ? nullptr : a.rope + int64_t(max(pos, 0)) * a.rope_dim;
    constexpr int kBatch = 8 / CH;  // heads whose loads are in flight together
    Turn turn[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) turn[c] = load_turn<MODE>(a, tab, min(4 * (lane + 32 * c), D - 4));
    for (int h0 = warp % per; h0 < a.q_heads; h0 += per * kBatch) {
        Raw raw[kBatch][CH];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                raw[i][c] = load_raw<T, MODE>(a, src + int64_t(min(h0 + i * per, a.q_heads - 1)) * D,
                                              min(4 * (lane + 32 * c), D - 4));
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int h = h0 + i * per, d = 4 * (lane + 32 * c);
                if (h >= a.q_heads || d >= D) continue;
                float y[4];
                turn4<T, MODE>(a, d, raw[i][c], turn[c], y);
                if (pos < 0) y[0] = y[1] = y[2] = y[3] = 0.f;
                *reinterpret_cast<uint2 *>(dst + int64_t(h) * D + d) =
                    make_uint2(act_t2<T>(y[0], y[1]), act_t2<T>(y[2], y[3]));
            }
    }
}

// RUNS: many tokens a sequence on average, and a block for each item and head of the long runs.  Else
// there mostly is no long run, so a few blocks look and, if there is one, take its items in turn.
template <typename T, bool F8, int CH, Mode MODE, bool RUNS>
__global__ void __launch_bounds__(kThreads, CH == 1 ? 3 : 2) kv_append_kernel(const __grid_constant__ AppendArgs a)
{
    grid_dep_launch();
    grid_dep_wait();  // the QKV projection and the batch's arrays may come from the kernel before
    // pages of long runs first, which take longest
    const int few_blocks = a.n_seqs * a.parts, pairs = 2 * a.c.kv_heads;
    int block = blockIdx.x;
    if (block < a.run_blocks) {
        if constexpr (RUNS) {
            append_item<T, F8, CH, MODE, RUNS>(a, block / pairs, block % pairs);
        } else {
#pragma unroll 1
            for (; block < a.items * pairs; block += a.run_blocks) {
                if (!append_item<T, F8, CH, MODE, RUNS>(a, block / pairs, block % pairs)) break;
                __syncthreads();  // the block's shared memory is read
            }
        }
        return;
    }
    block -= a.run_blocks;
    if (block < few_blocks) append_few<T, F8, CH, MODE>(a, block / a.parts, block % a.parts);
    else turn_queries<T, CH, MODE>(a, block - few_blocks);
}

template <typename T, bool F8, Mode MODE>
const void *append_kernel(bool wide, bool runs)
{
    if (runs)
        return wide ? reinterpret_cast<const void *>(kv_append_kernel<T, F8, 2, MODE, true>)
                    : reinterpret_cast<const void *>(kv_append_kernel<T, F8, 1, MODE, true>);
    return wide ? reinterpret_cast<const void *>(kv_append_kernel<T, F8, 2, MODE, false>)
                : reinterpret_cast<const void *>(kv_append_kernel<T, F8, 1, MODE, false>);
}

template <typename T, bool F8>
const void *append_kernel(Mode mode, bool wide, bool runs)
{
    switch (mode) {
    case kNone: return append_kernel<T, F8, kNone>(wide, runs);
    case kPairs: return append_kernel<T, F8, kPairs>(wide, runs);
    case kHalf: return append_kernel<T, F8, kHalf>(wide, runs);
    case kHalf2: return append_kernel<T, F8, kHalf2>(wide, runs);
    default: return append_kernel<T, F8, kAny>(wide, runs);
    }
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

wq_status check_kv(const wq_kv_cache *c, const wq_kv_batch *b, wq_dtype dt, int64_t M, int32_t q_heads)
{
    if (!c || !b) return fail(WQ_ERR_INVALID_ARG, "cache and batch must be non-null");
    if (dt != WQ_F16 && dt != WQ_BF16) return fail(WQ_ERR_INVALID_ARG, "dt must be WQ_F16 or WQ_BF16");
    if (M <= 0) return fail(WQ_ERR_INVALID_ARG, "M must be positive");
    if (c->format != WQ_FMT_INT && c->format != WQ_FMT_E4M3)
        return fail(WQ_ERR_INVALID_ARG, "cache format must be WQ_FMT_INT (INT8) or WQ_FMT_E4M3");
    if (c->num_pages <= 0) return fail(WQ_ERR_INVALID_ARG, "num_pages must be positive");
    if (c->page_size < kKvMinPage || c->page_size > kKvMaxPage || (c->page_size & (c->page_size - 1)))
        return fail(WQ_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (c->head_dim < 16 || c->head_dim > kKvMaxHeadDim || c->head_dim % 4)
        return fail(WQ_ERR_UNSUPPORTED, "head_dim must be a multiple of 4 from 16 to 256");
    if (c->kv_heads < 1 || c->kv_heads > 1024) return fail(WQ_ERR_INVALID_ARG, "kv_heads must be 1 .. 1024");
    if (c->num_pages > 0x7fffffff / int64_t(c->kv_heads)) return fail(WQ_ERR_INVALID_ARG, "num_pages * kv_heads exceeds int32");
    if (q_heads < 1 || q_heads % c->kv_heads) return fail(WQ_ERR_INVALID_ARG, "q_heads must be a multiple of kv_heads");
    if (M > 0x7fffffff / int64_t(q_heads)) return fail(WQ_ERR_INVALID_ARG, "M * q_heads exceeds int32");
    if (b->n_seqs < 1) return fail(WQ_ERR_INVALID_ARG, "n_seqs must be positive");
    if (b->n_seqs > kKvMaxSeqs) return fail(WQ_ERR_UNSUPPORTED, "n_seqs must be at most %d", kKvMaxSeqs);
    if (b->max_pages < 1 || b->max_pages > kKvMaxTokens / c->page_size)
        return fail(WQ_ERR_INVALID_ARG, "max_pages must be positive, and max_pages * page_size at most 2^31 - 1024");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !b->cu_q || !b->seq_len || !b->block_table)
        return fail(WQ_ERR_INVALID_ARG, "the pointers of cache and batch must be non-null");
    if (!aligned16(c->k) || !aligned16(c->v)) return fail(WQ_ERR_ALIGNMENT, "k and v must be 16-byte aligned");
    if (!aligned4(c->k_scale) || !aligned4(c->v_scale) || !aligned4(b->cu_q) || !aligned4(b->seq_len) ||
        !aligned4(b->block_table))
        return fail(WQ_ERR_ALIGNMENT, "scales and batch arrays must be 4-byte aligned");
    return WQ_OK;
}

}  // namespace wq

using namespace wq;

extern "C" wq_status kv_append(const void *qkv, wq_dtype dt, int64_t M, int32_t q_heads, const float *rope,
                               int64_t rope_len, int32_t rope_dim, int32_t rope_style, void *q_out,
                               const wq_kv_cache *cache, const wq_kv_batch *batch, cudaStream_t stream)
{
    wq_status rc = check_kv(cache, batch, dt, M, q_heads);
    if (rc != WQ_OK) return rc;
    if (!qkv || !q_out) return fail(WQ_ERR_INVALID_ARG, "qkv and q_out must be non-null");
    if ((rope != nullptr) != (rope_dim != 0)) return fail(WQ_ERR_INVALID_ARG, "rope is given with rope_dim > 0, or NULL with 0");
    if (rope_dim < 0 || rope_dim > cache->head_dim || rope_dim % 2)
        return fail(WQ_ERR_INVALID_ARG, "rope_dim must be even and at most head_dim");
    if (rope_style != WQ_ROPE_HALF && rope_style != WQ_ROPE_PAIRS) return fail(WQ_ERR_INVALID_ARG, "unknown rope_style");
    if (rope && rope_len < 1) return fail(WQ_ERR_INVALID_ARG, "rope_len must be positive");
    if (!aligned16(qkv) || !aligned16(q_out) || (rope && !aligned16(rope)))
        return fail(WQ_ERR_ALIGNMENT, "qkv, q_out and rope must be 16-byte aligned");

    AppendArgs a{};
    a.qkv = qkv;
    a.q_out = q_out;
    a.rope = rope;
    a.c = *cache;
    a.cu_q = batch->cu_q;
    a.seq_len = batch->seq_len;
    a.block_table = batch->block_table;
    a.n_seqs = int(batch->n_seqs);
    a.max_pages = int(batch->max_pages);
    a.M = int(M);
    a.q_heads = q_heads;
    a.rope_dim = rope_dim;
    while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
    a.pitch = kv_pitch(cache->head_dim);
    const int64_t capacity = batch->max_pages * cache->page_size;
    a.limit = int(rope ? std::min(capacity, rope_len) : capacity);
    a.pairs = rope_style == WQ_ROPE_PAIRS;
    // kHalf: partners and cos / sin at rope_dim / 2, a table row rope_dim values long; see Mode
    const Mode mode = !rope_dim                           ? kNone
                      : a.pairs                           ? (rope_dim % 4 == 0 ? kPairs : kAny)
                      : rope_dim % 8 == 0 ? kHalf
                      : rope_dim % 4 == 0 ? kHalf2 : kAny;
    // A page's rows go over all warps of a block for sequences that bring many tokens, else one warp
    // takes each (head, keys or values): 32 sequences of 8 tokens, 8 key heads, 7.1 us against 11.4 of
    // the former; 8 sequences of 16 tokens 12.1 against 4.9.
    a.parts = (2 * cache->kv_heads + kWarps - 1) / kWarps;
    // (a block an item with few tokens a sequence: 48 sequences of 1 to 6 tokens, 32 key heads, 12.3 us
    // instead of 8.1; one run of 380 tokens beside 127 of one: 18 us, 285 by a warp each)
    const bool runs = M > kKvFewTokens * batch->n_seqs;
    const int64_t items = M > kKvFewTokens ? kv_item_start(int(M), int(batch->n_seqs), a.page_shift, runs) : 0;
    const int64_t all = items * 2 * cache->kv_heads, run_blocks = runs ? all : std::min<int64_t>(all, device_info().sm_count);
    // Queries, a block a token or a warp a token: 1024 tokens of 32 heads 13.2 / 14.5 us, 1600 19.2 /
    // 19.5, 4096 48.5 / 39.3.  No more warps a token than heads: 256 tokens of one head 4.5 us with a
    // block each, 3.3 with a warp each, of four heads 4.8 and with two warps 3.8.
    int warps = 1;
    while (warps < kWarps && warps < q_heads) warps *= 2;
    a.q_tokens = M <= 1600 ? kWarps / warps : kWarps;
    const int64_t blocks = run_blocks + batch->n_seqs * a.parts + (M + a.q_tokens - 1) / a.q_tokens;
    if (std::max(all, blocks) > 0x7fffffff - device_info().sm_count)
        return fail(WQ_ERR_INVALID_ARG, "too many blocks: fewer rows or heads a call");
    a.items = int(items);
    a.run_blocks = int(run_blocks);
    const bool wide = cache->head_dim > 128, f8 = cache->format == WQ_FMT_E4M3;
    const void *fn = dt == WQ_F16 ? (f8 ? append_kernel<__half, true>(mode, wide, runs) : append_kernel<__half, false>(mode, wide, runs))
                                  : (f8 ? append_kernel<__nv_bfloat16, true>(mode, wide, runs)
                                        : append_kernel<__nv_bfloat16, false>(mode, wide, runs));
    PreparedLaunch L;
    L.set(fn, dim3(unsigned(blocks)), dim3(kThreads), 0, a);
    return launch_prepared(L, stream, "kv_append_kernel");
}
