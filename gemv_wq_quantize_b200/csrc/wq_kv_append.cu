// wq_kv_append.cu -- kv_append: rotary positions on the queries and keys of a fused QKV row,
// and the append of keys and values to a paged 8-bit cache, in one launch for sm_100a.
//
// Mathematics: a rotated pair is (a c - b s, b c + a s), every product and sum one binary32
// rounding; a page and head has one scale, max(scale before, max|x| * binary32(1 / qmax)) over the call's new
// tokens x of the page, and codes of x / scale.  A scale that grows re-codes the page's earlier
// tokens by (scale before / scale).
//
// Work items.  The maximum over a page's new tokens needs one owner per (page, head): a block
// owns one (sequence, page) item and a few heads.  Which sequence an item belongs to follows
// from cu_q alone (wq_kv.h), found by all threads of the block looking at once.  A group of WPT
// warps owns the keys or the values of one head: every lane holds four neighbouring values of a
// row (so the partner of a rotated value is one more 8-byte load of the same row, not a
// shuffle), the rows of the page go over the group's warps, and the rotated values stay in
// registers between the maximum and the codes.  Other blocks of the same launch turn the
// queries.
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
constexpr int kHeldFloats = 64;  // binary32 values of a page that a lane keeps in registers

struct AppendArgs {
    const void *qkv;
    void *q_out;
    const float *rope;
    wq_kv_cache c;
    const int32_t *cu_q, *seq_len, *block_table;
    int n_seqs, max_pages, M, q_heads;
    int rope_len, rope_dim;
    int page_shift, pitch;
    int capacity;       // tokens that the block table's row holds
    int limit;          // positions below it have a place: min(capacity, rope_len)
    bool pairs;         // WQ_ROPE_PAIRS
    bool vec;           // four neighbouring values turn alike and their partners are 8-byte aligned
    int64_t kv_items;   // (sequence, page) items
    int head_blocks;    // blocks per item
    int q_tokens;       // tokens of a query block
};

// Four neighbouring values d .. d + 3 of one head row, rotated by the position whose table row
// is `tab` (nullptr: not rotated).
template <typename T>
__device__ __forceinline__ void load_turned(const AppendArgs &a, const T *row, int d, const float *tab, float (&y)[4])
{
    const uint2 raw = *reinterpret_cast<const uint2 *>(row + d);
    const float2 lo = act_f2<T>(raw.x), hi = act_f2<T>(raw.y);
    const float x[4] = {lo.x, lo.y, hi.x, hi.y};
    const int r = a.rope_dim, half = r / 2;
    if (tab == nullptr || d >= r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[i];
    } else if (a.vec && a.pairs) {
        const float2 c = *reinterpret_cast<const float2 *>(tab + d / 2);
        const float2 s = *reinterpret_cast<const float2 *>(tab + half + d / 2);
        y[0] = __fsub_rn(__fmul_rn(x[0], c.x), __fmul_rn(x[1], s.x));
        y[1] = __fadd_rn(__fmul_rn(x[1], c.x), __fmul_rn(x[0], s.x));
        y[2] = __fsub_rn(__fmul_rn(x[2], c.y), __fmul_rn(x[3], s.y));
        y[3] = __fadd_rn(__fmul_rn(x[3], c.y), __fmul_rn(x[2], s.y));
    } else if (a.vec) {
        const bool first = d < half;
        const int u = first ? d : d - half;
        const uint2 praw = *reinterpret_cast<const uint2 *>(row + (first ? d + half : d - half));
        const float2 plo = act_f2<T>(praw.x), phi = act_f2<T>(praw.y);
        const float p[4] = {plo.x, plo.y, phi.x, phi.y};
        const float4 c = *reinterpret_cast<const float4 *>(tab + u);
        const float4 s = *reinterpret_cast<const float4 *>(tab + half + u);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float xc = __fmul_rn(x[i], cc[i]), ps = __fmul_rn(p[i], ss[i]);
            y[i] = first ? __fsub_rn(xc, ps) : __fadd_rn(xc, ps);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = d + i;
            if (e >= r) {
                y[i] = x[i];
                continue;
            }
            const bool first = a.pairs ? !(e & 1) : e < half;
            const int u = a.pairs ? e / 2 : (first ? e : e - half);
            const int partner = a.pairs ? (e ^ 1) : (first ? e + half : e - half);
            const float xc = __fmul_rn(x[i], tab[u]), ps = __fmul_rn(act_f(row[partner]), tab[half + u]);
            y[i] = first ? __fsub_rn(xc, ps) : __fadd_rn(xc, ps);
        }
    }
}

// The largest finite magnitude; NaN is stored as 0 (an infinity stays one, and saturates).
__device__ __forceinline__ float absmax_finite(float (&y)[4], float m)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (y[i] != y[i]) y[i] = 0.f;
        const float v = fabsf(y[i]);
        m = v <= FLT_MAX ? fmaxf(m, v) : m;
    }
    return m;
}

template <bool F8>
__device__ __forceinline__ uint32_t store_codes(float (&y)[4], float s, float r)
{
    // an infinity over a finite scale is the largest code
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (fabsf(y[i]) > FLT_MAX) y[i] = copysignf(FLT_MAX, y[i]);
    return codes4<F8>(y, s, r);
}

// Keys and values of one (sequence, page) item.  CH: chunks of 128 values of a head (a lane
// has four of each).
template <typename T, bool F8, int WPT, int CH>
__device__ __forceinline__ void append_item(const AppendArgs &a, int64_t item, int head_block)
{
    constexpr int kTasks = kWarps / WPT;  // (head, keys or values) pairs of the block
    constexpr int kHeld = kHeldFloats / (4 * CH);
    __shared__ int s_seq[4];
    __shared__ float s_max[kWarps];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) s_seq[0] = -1;
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1], len = a.seq_len[b];
        const int q0 = kv_clamp(lo, 0, a.M), q1 = kv_clamp(hi, q0, a.M);
        if (kv_item_start(q0, b, a.page_shift) <= item && item < kv_item_start(q1, b + 1, a.page_shift)) {
            s_seq[0] = b;
            s_seq[1] = lo;
            s_seq[2] = hi;
            s_seq[3] = len;
        }
    }
    __syncthreads();
    const int b = s_seq[0];
    if (b < 0) return;
    const KvSpan span = kv_span(s_seq[1], s_seq[2], s_seq[3], a.M, a.capacity);
    KvPageSpan ps = kv_page_span(span, item - kv_item_start(span.q0, b, a.page_shift), a.page_shift);
    if (ps.count == 0) return;
    const int pos0 = (ps.page << a.page_shift) + ps.off;
    const int count = min(ps.count, a.limit - pos0);  // positions beyond the rope table have no place
    const int64_t page = kv_page_ok(a.block_table[int64_t(b) * a.max_pages + ps.page], a.c.num_pages);
    if (tid == 0 && (page < 0 || count < ps.count || s_seq[3] > a.capacity))
        atomicCAS(&g_kv_append_error, kErrNone, kErrRange);
    if (page < 0 || count <= 0) return;

    const int task = warp / WPT, wi = warp % WPT;
    const int pair = head_block * kTasks + task;  // keys of head h, then its values
    const int head = pair / 2;
    const bool is_k = (pair & 1) == 0, live = head < a.c.kv_heads;
    const int D = a.c.head_dim;
    const int64_t row_stride = int64_t(a.q_heads + 2 * a.c.kv_heads) * D;
    const T *src = static_cast<const T *>(a.qkv) + int64_t(ps.token) * row_stride +
                   int64_t(a.q_heads + (is_k ? 0 : a.c.kv_heads) + head) * D;
    const float *tab = is_k && a.rope_dim ? a.rope + int64_t(pos0) * a.rope_dim : nullptr;
    float held[kHeld][CH][4];
    float amax = 0.f, before = 0.f;
    const int64_t si = kv_scale_index(page, head, a.c.kv_heads);
    float *scale = (is_k ? a.c.k_scale : a.c.v_scale) + si;
    if (live) {
        if (ps.off > 0) before = *scale;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int r = wi + i * WPT;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int d = 4 * (lane + 32 * c);
                if (r < count && d < D) {
                    load_turned<T>(a, src + r * row_stride, d, tab ? tab + int64_t(r) * a.rope_dim : nullptr, held[i][c]);
                    amax = absmax_finite(held[i][c], amax);
                }
            }
        }
        for (int r = wi + kHeld * WPT; r < count; r += WPT)
            for (int c = 0; c < CH; ++c) {
                const int d = 4 * (lane + 32 * c);
                if (d >= D) continue;
                float y[4];
                load_turned<T>(a, src + r * row_stride, d, tab ? tab + int64_t(r) * a.rope_dim : nullptr, y);
                amax = absmax_finite(y, amax);
            }
        amax = __uint_as_float(warp_umax(__float_as_uint(amax)));
    }
    if (WPT > 1) {
        if (lane == 0) s_max[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPT; ++i) amax = fmaxf(amax, s_max[task * WPT + i]);
    } else {
        __syncwarp();
    }
    if (!live) return;
    const float need = __fmul_rn(amax, kInvQmax<F8>);
    const float now = fmaxf(before, need);
    const float rnow = now != 0.f ? __frcp_rn(now) : 0.f;
    if (wi == 0 && lane == 0) *scale = now;
    uint8_t *codes = static_cast<uint8_t *>(is_k ? a.c.k : a.c.v) +
                     kv_code_offset(page, head, 0, a.c.kv_heads, a.page_shift, a.pitch);
    if (now > before && ps.off > 0) {  // the page's earlier tokens in the new scale
        const float ratio = __fdiv_rn(before, now);
        for (int r = wi; r < ps.off; r += WPT)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int d = 4 * (lane + 32 * c);
                if (d >= D) continue;
                uint32_t *p = reinterpret_cast<uint32_t *>(codes + int64_t(r) * a.pitch + d);
                const uint32_t w = *p;
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(code_value<F8>(w, i), ratio);
                *p = codes4<F8>(y, 1.f, 1.f);
            }
    }
    codes += int64_t(ps.off) * a.pitch;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int r = wi + i * WPT;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int d = 4 * (lane + 32 * c);
            if (r < count && d < D)
                *reinterpret_cast<uint32_t *>(codes + int64_t(r) * a.pitch + d) = store_codes<F8>(held[i][c], now, rnow);
        }
    }
    for (int r = wi + kHeld * WPT; r < count; r += WPT)
        for (int c = 0; c < CH; ++c) {
            const int d = 4 * (lane + 32 * c);
            if (d >= D) continue;
            float y[4];
            load_turned<T>(a, src + r * row_stride, d, tab ? tab + int64_t(r) * a.rope_dim : nullptr, y);
            absmax_finite(y, 0.f);
            *reinterpret_cast<uint32_t *>(codes + int64_t(r) * a.pitch + d) = store_codes<F8>(y, now, rnow);
        }
}

// The queries of q_tokens tokens: kWarps / q_tokens warps take a token's heads in turn.
template <typename T, int CH>
__device__ __forceinline__ void turn_queries(const AppendArgs &a, int64_t block)
{
    __shared__ int s_pos[kWarps];  // position; -1: no place; -2: not part of a sequence
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t m0 = block * a.q_tokens;
    if (tid < kWarps) s_pos[tid] = -2;
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int len = a.seq_len[b];
        const KvSpan s = kv_span(a.cu_q[b], a.cu_q[b + 1], len, a.M, a.capacity);
        for (int64_t m = max(int64_t(s.q0), m0); m < min(int64_t(s.q0) + s.n, m0 + a.q_tokens); ++m) {
            const int p = s.len - s.n + int(m - s.q0);
            s_pos[m - m0] = p < 0 || p >= a.limit ? -1 : p;
            if (p >= a.limit || len > a.capacity) atomicCAS(&g_kv_append_error, kErrNone, kErrRange);
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
    const float *tab = a.rope_dim && pos >= 0 ? a.rope + int64_t(pos) * a.rope_dim : nullptr;
    for (int h = warp % per; h < a.q_heads; h += per)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int d = 4 * (lane + 32 * c);
            if (d >= D) continue;
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            if (pos >= 0) load_turned<T>(a, src + int64_t(h) * D, d, tab, y);
            *reinterpret_cast<uint2 *>(dst + int64_t(h) * D + d) = make_uint2(act_t2<T>(y[0], y[1]), act_t2<T>(y[2], y[3]));
        }
}

template <typename T, bool F8, int WPT, int CH>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendArgs a)
{
    grid_dep_launch();
    grid_dep_wait();  // the QKV projection and the batch's arrays may come from the kernel before
    const int64_t kv_blocks = a.kv_items * a.head_blocks;
    if (int64_t(blockIdx.x) < kv_blocks)
        append_item<T, F8, WPT, CH>(a, blockIdx.x / a.head_blocks, blockIdx.x % a.head_blocks);
    else
        turn_queries<T, CH>(a, blockIdx.x - kv_blocks);
}

template <typename T, bool F8>
const void *append_kernel(bool many, bool wide)
{
    if (many)
        return wide ? reinterpret_cast<const void *>(kv_append_kernel<T, F8, 4, 2>)
                    : reinterpret_cast<const void *>(kv_append_kernel<T, F8, 4, 1>);
    return wide ? reinterpret_cast<const void *>(kv_append_kernel<T, F8, 1, 2>)
                : reinterpret_cast<const void *>(kv_append_kernel<T, F8, 1, 1>);
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
    if (c->num_pages <= 0 || c->num_pages > 0x7fffffff) return fail(WQ_ERR_INVALID_ARG, "num_pages must be 1 .. 2^31 - 1");
    if (c->page_size < kKvMinPage || c->page_size > kKvMaxPage || (c->page_size & (c->page_size - 1)))
        return fail(WQ_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (c->head_dim < 16 || c->head_dim > kKvMaxHeadDim || c->head_dim % 4)
        return fail(WQ_ERR_UNSUPPORTED, "head_dim must be a multiple of 4 from 16 to 256");
    if (c->kv_heads < 1 || c->kv_heads > 1024) return fail(WQ_ERR_INVALID_ARG, "kv_heads must be 1 .. 1024");
    if (q_heads < 1 || q_heads % c->kv_heads) return fail(WQ_ERR_INVALID_ARG, "q_heads must be a multiple of kv_heads");
    if (M > 0x7fffffff / int64_t(q_heads)) return fail(WQ_ERR_INVALID_ARG, "M * q_heads exceeds int32");
    if (b->n_seqs < 1) return fail(WQ_ERR_INVALID_ARG, "n_seqs must be positive");
    if (b->n_seqs > kKvMaxSeqs) return fail(WQ_ERR_UNSUPPORTED, "n_seqs must be at most %d", kKvMaxSeqs);
    if (b->max_pages < 1 || b->max_pages > 0x7fffffff / c->page_size)
        return fail(WQ_ERR_INVALID_ARG, "max_pages must be positive, and max_pages * page_size below 2^31");
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
    a.capacity = int(batch->max_pages * cache->page_size);
    a.limit = rope ? int(std::min<int64_t>(a.capacity, rope_len)) : a.capacity;
    a.pairs = rope_style == WQ_ROPE_PAIRS;
    // WQ_ROPE_HALF: a value's partner is rope_dim / 2 away, and its four cos / sin lie at that
    // multiple too; a table row is rope_dim values long
    a.vec = a.pairs ? rope_dim % 4 == 0 : rope_dim % 8 == 0;
    a.kv_items = (M >> a.page_shift) + 2 * batch->n_seqs;
    // A page's rows go over four warps where sequences bring many tokens, else one warp takes
    // each (head, keys or values).
    const bool many = M >= 4 * batch->n_seqs;
    a.head_blocks = many ? cache->kv_heads : (cache->kv_heads + 3) / 4;
    a.q_tokens = M <= 1024 ? 1 : kWarps;
    const int64_t blocks = a.kv_items * a.head_blocks + (M + a.q_tokens - 1) / a.q_tokens;
    if (blocks > 0x7fffffff) return fail(WQ_ERR_INVALID_ARG, "too many blocks: fewer rows or heads a call");
    const bool wide = cache->head_dim > 128, f8 = cache->format == WQ_FMT_E4M3;
    const void *fn = dt == WQ_F16 ? (f8 ? append_kernel<__half, true>(many, wide) : append_kernel<__half, false>(many, wide))
                                  : (f8 ? append_kernel<__nv_bfloat16, true>(many, wide)
                                        : append_kernel<__nv_bfloat16, false>(many, wide));
    PreparedLaunch L;
    L.set(fn, dim3(unsigned(blocks)), dim3(kThreads), 0, a);
    return launch_prepared(L, stream, "kv_append_kernel");
}
