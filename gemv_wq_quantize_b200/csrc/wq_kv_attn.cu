// wq_kv_attn.cu -- kv_attention: the C entry points, and the kernel for few rows per key head
// (decode and draft verification): attention over the paged 8-bit cache, split over the whole
// GPU by key ranges, on the 5th-generation tensor cores (tcgen05) without widening a code.
//
// Mathematics: for a query row q of position p and the keys j <= p of its sequence,
//   s_j = sm_scale * ks[page(j)] * (q . kc_j),   out = sum_j softmax(s)_j vs[page(j)] vc_j
// with a running maximum and sum, and the two page scales applied in binary32.
//
// Bound by reading the cache once; widening the codes to binary16 in registers took 850
// instructions a warp for 32 keys and held the reads to 4.7 TB/s.  So the codes are MMA operands as
// they lie in memory, and the few rows are cut into 8-bit parts instead:
//   q = 2^e (q1 + q2 / 16 + q3 / 256 + q4 / 4096)      e4m3 cache: each part the e4m3 value nearest
//                                                       to what is left
//   q = 2^e (q1 2^21 + q2 2^14 + q3 2^7 + q4)           INT8 cache: digits of a 28-bit integer
// (exact for binary16 and bfloat16 down to 2^-27 of the row's largest value), and the weights times
// their value scales likewise: over a power of two that is at most twice the largest scale so far, to
// 2^-27 (INT8), or to 2^-16 of each and 2^-28 (e4m3).  The parts of all rows are the N side of both
// products,
//   S^T[key][part, row] = K Q^T      A = 128 keys of codes (rows of dimensions),
//   O^T[dimension][part, row] = V^T P^T      A = the values of 128 keys, read dimension-major,
// with binary32 (e4m3) or exact int32 (INT8) accumulators in Tensor Memory, and the parts are put
// together in binary32 when a step's scores or sums are read back.
//  * warps 0-3: a thread per key for the softmax (maxima over the warps through shared memory),
//    and a thread per dimension for the output, which is added up in registers step by step;
//  * warp 4: one thread issues the MMAs, the next step's scores in front of this step's sums;
//  * warp 5: fills a ring of stages of 128 keys and values by TMA, page by page, and their scales.
// Every wait is bounded; on expiry the block records an error, stops and frees its Tensor Memory.
//
// Work split: tiles (sequence, key head, 8 rows) are cut into units of 128 keys, and the
// persistent blocks take equal contiguous shares of all units, whatever the lengths (a tile counts
// kTileUnits more, about what its start and end take).  A tile cut over several blocks leaves
// partial sums in the workspace; the last block to arrive adds them in the order of their keys,
// so the result does not depend on which block that is.
//
// Measured (device time, calls back to back in a graph), 32 query heads: two sequences of 131000 keys, 8
// key heads of 128: 93 us, 5.8 TB/s (99 us each, 5.4 TB/s, by a caller's clock); 32 of 100 to 4095 keys:
// 40 us, 3.4 TB/s, with heads of 256 64 us; 16 of 2 to 6 tokens and 300 to 2000 keys, 32 key heads of 100:
// 49.5 us, 2.2 TB/s; one of 512 keys, 32 key heads: 14 us, where a block's start (Tensor Memory, shares,
// queries), one to five steps and the joining of the parts follow one another.
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "wq_act.cuh"
#include "wq_kv_attn.cuh"
#include "wq_tc.cuh"

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

constexpr int kKeys = 128;               // keys of a step: MMA M of the scores
constexpr int kGroups = kKeys / 16;      // a group of 16 keys lies in one page
constexpr int kSoft = 128;               // threads of the softmax warps
constexpr int kMmaWarp = 4, kCopyWarp = 5, kThreads = 192;
constexpr int kParts = 4;                // 8-bit parts of a query value or weight
constexpr int kUnitShift = 7;            // a unit: 128 keys, the granule of the split
constexpr int kTileUnits = 4;            // what the start and end of a tile cost a block, in units
constexpr int kLeastUnits = 1;           // of a share, beside them: more leaves SMs idle at short lengths
constexpr int kMostUnits = 0x7fffff00;   // of a call

__device__ __forceinline__ uint64_t globaltimer()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Rows of a tile.  16 (and a stage less in the ring) measured slower even where a sequence has more, whose
// keys are then read again from L2: 16 sequences of 2000 keys and 16 rows 43 / 50 us, two of 8000 keys
// and 96 rows 71 / 78.
constexpr int kRowsOfTile = 8;

// NB: boxes of 128 dimensions (1 up to a head size of 128, 2 up to 256).  NR: rows of a tile.
template <int NB, int NR>
struct Shape {
    static constexpr int kN = kParts * NR;               // MMA N
    static constexpr int kBox = kKeys * 128;             // bytes of 128 keys x 128 dimensions
    static constexpr int kPerSm = NB == 1 ? 2 : 1;       // blocks
    static constexpr int kStages = 3;                    // 96 KB (192 KB) of a block's share of an SM
    static constexpr int kRowFloats = 128 * NB + 4;      // a partial row: sums, maximum, weight sum
    static constexpr uint32_t kSCol = 0, kOCol = 2 * kN; // two of each: scores [2], sums [2][NB]
    static constexpr uint32_t kUsed = 2 * kN * (1 + NB), kTmem = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
};

template <int NB, int NR>
struct Smem {
    using S = Shape<NB, NR>;
    alignas(1024) uint8_t k[S::kStages][NB][S::kBox];
    alignas(1024) uint8_t v[S::kStages][NB][S::kBox];
    alignas(1024) uint8_t q[NB][S::kN * 128];  // rows (part, row) of 128 dimensions
    alignas(1024) uint8_t p[2][S::kN * 128];   // rows (part, row) of 128 keys
    uint64_t full[S::kStages], empty[S::kStages], scales[S::kStages], s_full[2], p_full[2], o_full[2], q_full, joined;
    float ks[S::kStages][kGroups], vs[S::kStages][kGroups], v_max[S::kStages];
    uint32_t dead[S::kStages];   // groups whose block-table entry is no page
    float q_scale[NR];           // of a row's parts, times sm_scale and log2 e
    int seen[NR];                // keys that a row sees (0: no row)
    int64_t row_at[NR];          // its first element in q and out
    alignas(16) int top[2][NR][4];    // the warps' maxima of a step (order_of)
    float sum[4][NR];            // the warps' weight sums of a tile
    int64_t units[kThreads / 32];
    int first[2], parts[2];      // the tiles that this block left partials of
    int abort;
    uint32_t tmem;
    int before[1];               // the units of all sequences before each: n_seqs + 1
};

// A bounded wait: about 2 s, or `after` (nanoseconds) once another role gave up.  wait_warp: one
// answer for the warp.  The softmax warps go on after a wait that gave up, so that they reach the
// same barriers as often; what they then write is not valid.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t after = 100000)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait_short(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_short(bar, parity)) return true;
        if (globaltimer() - t0 > (*abort ? after : 2000000000ull)) {
            atomicCAS(&g_kv_attn_error, kErrNone, kErrWaitTimeout);
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t after = 100000)
{
    return __all_sync(0xffffffffu, wait(bar, parity, abort, after));
}

template <bool F8>
__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (F8) tc::mma_f8_ss(d, a, b, idesc, accumulate);
    else tc::mma_i8_ss(d, a, b, idesc, accumulate);
}

// The parts of four values x (e4m3: |x| < 448, each part the value nearest to sixteen times what
// the ones before left; INT8: x an integer below 2^28 in magnitude, 7 bits a digit, the first with
// the sign), as bytes of a word per part.
template <bool F8>
__device__ __forceinline__ void split4(const float (&x)[4], uint32_t (&part)[kParts])
{
    if constexpr (F8) {
        float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const uint32_t w = e4m3x4(r[0], r[1], r[2], r[3]);
            part[p] = w;
            if (p + 1 < kParts)
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = (r[i] - code_value<true>(w, i)) * 16.f;
        }
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = uint32_t(__float2int_rn(x[i]));
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = p == 0 ? uint32_t(int32_t(u[i]) >> 21) : (u[i] >> (21 - 7 * p)) & 127u;
            part[p] = prmt(prmt(b[0], b[1], 0x0040), prmt(b[2], b[3], 0x0040), 0x5410);
        }
    }
}
// The value of accumulated parts, in units of the first (e4m3) or the last (INT8).
template <bool F8>
__device__ __forceinline__ float whole_of(uint32_t c1, uint32_t c2, uint32_t c3, uint32_t c4)
{
    if constexpr (F8)
        return fmaf(fmaf(fmaf(__uint_as_float(c4), 0.0625f, __uint_as_float(c3)), 0.0625f, __uint_as_float(c2)), 0.0625f,
                    __uint_as_float(c1));
    else
        return fmaf(float(int(c1)), 2097152.f, fmaf(float(int(c2)), 16384.f, fmaf(float(int(c3)), 128.f, float(int(c4)))));
}
// Exponents: a query row with largest value 2^e .. 2^(e+1) is multiplied by 2^(kQUp - e) before it
// is cut; a weight, at most 2^kSlack and under its reference's value scale, by kPUp (to at most
// 256, or 2^28).  A maximum that rises by less than kSlack is not followed.
constexpr float kSlack = 2.f;
template <bool F8>
constexpr int kQUp = F8 ? 7 : 26;
template <bool F8>
constexpr float kPUp = F8 ? 64.f : 67108864.f;

// A power of two's inverse (normal, and so is the inverse).
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// Whether any thread of the softmax warps has the predicate: their barrier and the answer in one.
__device__ __forceinline__ bool soft_any(bool mine)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(uint32_t(mine)), "n"(kSoft)
        : "memory");
    return any != 0;
}

// Signed integers in the order of the floats (NaN above all), for the warp-wide integer maximum.
__device__ __forceinline__ int order_of(float x)
{
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_order(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

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
    t.s = kv_span(a.cu_q[lo], a.cu_q[lo + 1], a.seq_len[lo], a.M, a.capacity);
    const bool split = a.partials != nullptr;
    const int head_units = split ? kTileUnits : 0;
    const int units = split ? head_units + kv_units(t.s.len, shift) : 1;
    const int tiles = int(kv_tiles(t.s.n, a.group, ROWS));
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

__device__ __forceinline__ uint16_t *out_row(const KvAttnArgs &a, const Tile &t, int r)
{
    const int row = t.row0 + r;
    return static_cast<uint16_t *>(a.out) +
           (int64_t(t.s.q0 + row / a.group) * a.q_heads + t.head * a.group + row % a.group) * a.head_dim;
}
__device__ __forceinline__ float inverse_of(float l) { return l > 0.f ? 1.f / l : (l == l ? 0.f : l); }
__device__ __forceinline__ float weight_of(float m, float top) { return m == -INFINITY ? 0.f : exp2_approx(m - top); }

// A block's share of the units: its parts of tiles, one after the other (every role walks them).
template <int NR>
struct Share {
    const KvAttnArgs &a;
    const int *before;
    int shift, u, u_end;
    __device__ __forceinline__ bool next(Tile &t)
    {
        while (u < u_end) {
            int behind;
            t = tile_of<NR>(a, before, shift, u, u_end, behind);
            u = behind;
            if (behind > t.u0) return true;  // (else none of the tile's keys)
        }
        return false;
    }
};
__device__ __forceinline__ int steps_of(const Tile &t) { return (t.t1 - t.t0 + kKeys - 1) / kKeys; }

// ------------------------------------------------------------------ codes and scales of the steps
// A step's keys and values arrive as one box per page part and 128 dimensions (zeros behind the
// head).  Lanes 0 .. 7 look up a box's page, lanes 8 .. 15 a group's, and its scales, which go out
// one step later, so that copies do not wait for them.
template <int NB, int NR>
__device__ __forceinline__ void copy_role(const KvAttnArgs &a, const CUtensorMap *km, const CUtensorMap *vm, Smem<NB, NR> &sm,
                                          Share<NR> share)
{
    using S = Shape<NB, NR>;
    const int lane = threadIdx.x % 32;
    const int box_rows = min(1 << a.page_shift, kKeys), boxes = kKeys / box_rows;
    const int my_key = lane < kGroups ? lane * box_rows : (lane - kGroups) * 16;
    const bool boxed = lane < boxes, grouped = lane >= kGroups && lane < 2 * kGroups;
    uint32_t step = 0;
    float ks = 0.f, vs = 0.f;
    bool bad = false, pending = false, ok = true;
    auto publish = [&]() {  // the scales of step - 1
        if (!pending) return;
        const int slot = (step - 1) % S::kStages;
        const uint32_t dead = __ballot_sync(0xffffffffu, bad) >> kGroups;
        const float top = __uint_as_float(warp_umax(__float_as_uint(fabsf(vs))));
        if (grouped) {
            sm.ks[slot][lane - kGroups] = ks;
            sm.vs[slot][lane - kGroups] = vs;
        }
        if (lane == 0) {
            sm.dead[slot] = dead;
            sm.v_max[slot] = top;
            if (dead) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.scales[slot]);
        pending = false;
    };
    Tile t;
    while (ok && share.next(t)) {
        const int32_t *table = a.block_table + int64_t(t.b) * a.max_pages;
        auto entry_of = [&](int key) { return (boxed || grouped) && key < t.t1 ? table[key >> a.page_shift] : 0; };
        const int n = steps_of(t);
        int entry = n ? entry_of(t.t0 + my_key) : 0;
        for (int j = 0; j < n; ++j) {
            const int key = t.t0 + j * kKeys + my_key, slot = step % S::kStages;
            const uint32_t round = step / S::kStages;
            const bool used = (boxed || grouped) && key < t.t1;
            const int64_t page = used ? kv_page_ok(entry, a.num_pages) : -1;
            const int z = page < 0 ? -1 : int(page) * a.kv_heads + t.head;
            const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, boxed && z >= 0))) * uint32_t(box_rows * 128 * NB);
            const int y = key & ((1 << a.page_shift) - 1);
            if (round && !wait_warp(&sm.empty[slot], (round - 1) & 1, &sm.abort)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], 2 * bytes);
            __syncwarp();
            if (boxed && z >= 0)
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    tma_load_3d(sm.k[slot][c] + lane * box_rows * 128, km, 128 * c, y, z, &sm.full[slot]);
                    tma_load_3d(sm.v[slot][c] + lane * box_rows * 128, vm, 128 * c, y, z, &sm.full[slot]);
                }
            publish();
            ks = grouped && z >= 0 ? a.k_scale[z] : 0.f;
            vs = grouped && z >= 0 ? a.v_scale[z] : 0.f;
            bad = grouped && used && z < 0;
            pending = true;
            ++step;
            if (j + 1 < n) entry = entry_of(key + kKeys);
        }
    }
    publish();
    // nothing may land in shared memory after the block exits
    for (uint32_t i = step > uint32_t(S::kStages) ? step - S::kStages : 0; i < step; ++i)
        wait_warp(&sm.full[i % S::kStages], (i / S::kStages) & 1, &sm.abort, 20000000);
}

// ------------------------------------------------------------------ MMA issue (one thread)
template <bool F8, int NB, int NR>
__device__ __forceinline__ void mma_role(const KvAttnArgs &a, Smem<NB, NR> &sm, Share<NR> share, uint32_t tbase, uint64_t *fin)
{
    using S = Shape<NB, NR>;
    const uint32_t kmajor = F8 ? tc::idesc_f8(kKeys, S::kN) : tc::idesc_i8(kKeys, S::kN);
    const uint32_t iqk = kmajor, ipv = kmajor | tc::kIdescATransposed;
    const uint64_t dk = tc::sdesc_sw128(smem_u32(sm.k)), dv = tc::sdesc_sw128(smem_u32(sm.v));
    const uint64_t dq = tc::sdesc_sw128(smem_u32(sm.q)), dp = tc::sdesc_sw128(smem_u32(sm.p));
    // the scores of a step: 32 dimensions an MMA
    auto qk = [&](uint32_t step) {
        const uint64_t k = dk + uint64_t((step % S::kStages) * (NB * S::kBox) >> 4);
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_8bit<F8>(tbase + S::kSCol + (step & 1) * S::kN, k + uint64_t((c * S::kBox + i * 32) >> 4),
                             dq + uint64_t((c * S::kN * 128 + i * 32) >> 4), iqk, c + i > 0);
        tc::commit(&sm.s_full[step & 1]);
    };
    // the sums of a step: 32 keys an MMA; A is dimension-major: 128 bytes of dimensions a key, groups
    // of 8 keys 1024 bytes apart
    auto pv = [&](uint32_t step) {
        const uint64_t v = dv + uint64_t((step % S::kStages) * (NB * S::kBox) >> 4);
        const uint64_t p = dp + uint64_t((step & 1) * (S::kN * 128) >> 4);
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_8bit<F8>(tbase + S::kOCol + ((step & 1) * NB + c) * S::kN, v + uint64_t((c * S::kBox + i * 4096) >> 4),
                             p + uint64_t((i * 32) >> 4), ipv, i > 0);
        tc::commit(&sm.o_full[step & 1]);
        tc::commit(&sm.empty[step % S::kStages]);
    };
    uint32_t step = 0, queries = 0;
    Tile t;
    bool ok = true;
    auto scores_of = [&](uint32_t s) {
        if (!wait(&sm.full[s % S::kStages], (s / S::kStages) & 1, &sm.abort)) return false;
        tc::fence_after_sync();
        qk(s);
        return true;
    };
    while (ok && share.next(t)) {
        const int n = steps_of(t);
        if (n == 0) continue;
        ok = wait(&sm.q_full, queries++ & 1, &sm.abort) && scores_of(step);
        for (int j = 0; j < n && ok; ++j, ++step) {
            ok = (j + 1 == n || scores_of(step + 1)) && wait(&sm.p_full[step & 1], (step >> 1) & 1, &sm.abort);
            if (!ok) break;
            tc::fence_after_sync();
            pv(step);
        }
    }
    tc::commit(fin);  // all MMAs complete before the Tensor Memory is freed
    wait(fin, 0, &sm.abort, 20000000);
}

// ------------------------------------------------------------------ softmax and output
// Where the tile's rows are and what they see, by NR threads.
template <int NB, int NR>
__device__ __forceinline__ void place_rows(const KvAttnArgs &a, Smem<NB, NR> &sm, const Tile &t)
{
    const int r = threadIdx.x, row = t.row0 + r;
    if (r >= NR) return;
    const int i = r < t.rows ? row / a.group : 0, h = r < t.rows ? row % a.group : 0;
    sm.row_at[r] = (int64_t(t.s.q0 + i) * a.q_heads + t.head * a.group + h) * a.head_dim;
    sm.seen[r] = r < t.rows ? min(t.t1, t.s.len - t.s.n + i + 1) : 0;
}

// Rows [0, NR) of the tile to shared memory as parts, sixteen threads a row.
template <bool F8, bool BF16, int NB, int NR>
__device__ __forceinline__ void cut_queries(const KvAttnArgs &a, Smem<NB, NR> &sm, const Tile &t)
{
    using S = Shape<NB, NR>;
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    const int tid = threadIdx.x, x16 = tid % 16;
#pragma unroll 1
    for (int r = tid / 16; r < NR; r += kSoft / 16) {
        const bool live = r < t.rows;
        const uint16_t *q = static_cast<const uint16_t *>(a.q) + sm.row_at[r];
        uint2 raw[NB][2];
        uint32_t amax = 0;
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int d = 128 * c + 8 * x16 + 4 * h;
                raw[c][h] = live && d < a.head_dim ? *reinterpret_cast<const uint2 *>(q + d) : make_uint2(0, 0);
                const float2 lo = act_f2<T>(raw[c][h].x), hi = act_f2<T>(raw[c][h].y);
                // (as bit patterns: infinities and NaN are the largest)
                amax = max(max(max(amax, __float_as_uint(fabsf(lo.x))), max(__float_as_uint(fabsf(lo.y)), __float_as_uint(fabsf(hi.x)))),
                           __float_as_uint(fabsf(hi.y)));
            }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = kv_clamp(int(amax >> 23) - 127, -90, 120);
        const float up = __uint_as_float(uint32_t(127 + kQUp<F8> - e) << 23);
        const float down = __uint_as_float(uint32_t(127 + e - kQUp<F8>) << 23);
        if (x16 == 0) sm.q_scale[r] = amax < 0x7f800000u ? down * (a.sm_scale * kLog2e) : __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            uint32_t part[2][kParts];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 lo = act_f2<T>(raw[c][h].x), hi = act_f2<T>(raw[c][h].y);
                const float x[4] = {lo.x * up, lo.y * up, hi.x * up, hi.y * up};
                split4<F8>(x, part[h]);
            }
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const int n = p * NR + r;
                *reinterpret_cast<uint2 *>(sm.q[c] + n * 128 + (((x16 / 2) ^ (n & 7)) << 4) + 8 * (x16 % 2)) =
                    make_uint2(part[0][p], part[1][p]);
            }
        }
    }
}

// The block's part of a tile: scores, weights and sums step by step; `step` counts over all tiles.
template <int NB, int NR>
struct State {
    float o[NB][NR];  // of the thread's dimension(s), over vref
    float m[NR], l[NR], vref;  // l: of the thread's keys
};

template <bool F8, int NB, int NR>
__device__ __forceinline__ void add_sums(Smem<NB, NR> &sm, uint32_t step, uint32_t tlane, const float (&f)[NR], State<NB, NR> &st)
{
    using S = Shape<NB, NR>;
    wait_warp(&sm.o_full[step & 1], (step >> 1) & 1, &sm.abort);
    tc::fence_after_sync();
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int h = 0; h < NR / 8; ++h) {
            uint32_t x[kParts][8];
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                tc::ld_32x32b_x8(tlane + S::kOCol + ((step & 1) * NB + c) * S::kN + p * NR + 8 * h, x[p]);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * h + i;
                st.o[c][r] = fmaf(whole_of<F8>(x[0][i], x[1][i], x[2][i], x[3][i]), 1.f / kPUp<F8>, st.o[c][r] * f[r]);
            }
        }
}

template <bool F8, int NB, int NR>
__device__ __forceinline__ void attend(const KvAttnArgs &a, Smem<NB, NR> &sm, const Tile &t, uint32_t &step, uint32_t tbase,
                                       State<NB, NR> &st)
{
    using S = Shape<NB, NR>;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, n = steps_of(t);
    const uint32_t tlane = tbase + (uint32_t(32 * warp) << 16);
    const int least = sm.seen[0];  // keys that every row sees
    float f[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) f[r] = 1.f;
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++step) {
        const int slot = step % S::kStages, b = step & 1, key0 = t.t0 + j * kKeys, key = key0 + tid;
        wait_warp(&sm.scales[slot], (step / S::kStages) & 1, &sm.abort);
        wait_warp(&sm.s_full[b], (step >> 1) & 1, &sm.abort);
        tc::fence_after_sync();
        const uint32_t dead = sm.dead[slot];
        const bool gone = key >= t.t1 || (dead >> (tid / 16) & 1);
        const bool masked = key0 + kKeys > least || dead;
        const float ks = sm.ks[slot][tid / 16];
        float s[NR];
#pragma unroll
        for (int h = 0; h < NR / 8; ++h) {
            uint32_t x[kParts][8];
#pragma unroll
            for (int p = 0; p < kParts; ++p) tc::ld_32x32b_x8(tlane + S::kSCol + b * S::kN + p * NR + 8 * h, x[p]);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * h + i;
                s[r] = whole_of<F8>(x[0][i], x[1][i], x[2][i], x[3][i]) * (ks * sm.q_scale[r]);
            }
        }
        if (masked)
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (gone || key >= sm.seen[r]) s[r] = -INFINITY;
        // ---- new references where a score rose too far over the maximum so far (or is the first), or
        // a larger value scale arrived
        float f_now[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) f_now[r] = 1.f;
        const float vmax = sm.v_max[slot];
        bool rose = vmax >= st.vref && vmax > 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r) rose |= !(s[r] <= __fadd_rd(st.m[r], kSlack));  // (NaN too; rounded up it may be m + 4)
        if (soft_any(rose)) {
            int mine = 0;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int top = __reduce_max_sync(0xffffffffu, order_of(s[r]));
                if (lane == r) mine = top;
            }
            if (lane < NR) sm.top[b][lane][warp] = mine;
            named_bar_sync(1, kSoft);
            float fv = 1.f;
            if (vmax >= st.vref && vmax > 0.f) {
                const float vnew = __uint_as_float((__float_as_uint(fmaxf(vmax, 0x1p-120f)) & 0x7f800000u) + 0x00800000u);
                fv = st.vref * inverse_pow2(vnew);
                st.vref = vnew;
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int4 x = *reinterpret_cast<const int4 *>(sm.top[b][r]);
                const float m = of_order(max(max(max(x.x, x.y), max(x.z, x.w)), order_of(st.m[r])));
                const float fm = m == st.m[r] ? 1.f : exp2_approx(st.m[r] - m);
                st.m[r] = m;
                st.l[r] *= fm;
                f_now[r] = fm * fv;
            }
        }
        // (the scale over vref first, which is below 1: 2^26 / vref may be beyond binary32)
        const float v = gone || st.vref == 0.f ? 0.f : sm.vs[slot][tid / 16] * inverse_pow2(st.vref) * kPUp<F8>;
        float w[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            w[r] = s[r] == -INFINITY ? 0.f : exp2_approx(s[r] - st.m[r]);
            st.l[r] += w[r];
        }
        // ---- the weights' parts: a byte per (part, row), this thread's key
        uint8_t *pb = sm.p[b];
#pragma unroll
        for (int r0 = 0; r0 < NR; r0 += 4) {
            const float x[4] = {w[r0] * v, w[r0 + 1] * v, w[r0 + 2] * v, w[r0 + 3] * v};
            uint32_t part[kParts];
            split4<F8>(x, part);
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = p * NR + r0 + i;
                    pb[row * 128 + (((tid / 16) ^ (row & 7)) << 4) + tid % 16] = uint8_t(part[p] >> (8 * i));
                }
        }
        if (F8 && gone) {  // slots without a key may hold NaN codes, which a weight of 0 does not silence
#pragma unroll 1
            for (int c = 0; c < NB * 8; ++c) sts128(sm.v[slot][c / 8] + tid * 128 + c % 8 * 16, make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
        // ---- the sums of the step before, while this one's are on their way
        if (j > 0) add_sums<F8, NB, NR>(sm, step - 1, tlane, f, st);
#pragma unroll
        for (int r = 0; r < NR; ++r) f[r] = f_now[r];
    }
    if (n) add_sums<F8, NB, NR>(sm, step - 1, tlane, f, st);
}

// The finished rows of a tile, or this block's partial in `slot`.
template <typename T, int NB, int NR>
__device__ __forceinline__ void finish(const KvAttnArgs &a, Smem<NB, NR> &sm, const Tile &t, State<NB, NR> &st, float *slot)
{
    using S = Shape<NB, NR>;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float l = st.l[r];
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == r) mine = l;
    }
    if (lane < NR) sm.sum[warp][lane] = mine;
    named_bar_sync(1, kSoft);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        if (r >= t.rows) break;
        const float l = sm.sum[0][r] + sm.sum[1][r] + sm.sum[2][r] + sm.sum[3][r];
        const float inv = slot ? 1.f : inverse_of(l);  // (before vref: vref / l may be below the normal numbers)
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            const int d = 128 * c + tid;
            const float x = st.vref > 0.f ? st.o[c][r] * inv * st.vref : (l == l ? 0.f : l);
            if (slot) slot[r * S::kRowFloats + d] = x;
            else if (d < a.head_dim) static_cast<T *>(a.out)[sm.row_at[r] + d] = act_t<T>(x);
        }
        if (slot && tid == 0) *reinterpret_cast<float2 *>(slot + r * S::kRowFloats + 128 * NB) = make_float2(st.m[r], l);
    }
    named_bar_sync(1, kSoft);  // the sums are read
}

// Joins the partials of a tile: those of `parts` blocks from p0 on (its second slot, the others'
// first), in the order of their keys.  They come to the ring's memory in one go; `round` counts the
// waits on sm.joined.
template <typename T, int NB, int NR>
__device__ __forceinline__ void join_parts(const KvAttnArgs &a, Smem<NB, NR> &sm, const Tile &t, const float *p0, int parts,
                                           uint32_t &round)
{
    using S = Shape<NB, NR>;
    constexpr int kQuads = 32 * NB, kSlot = NR * S::kRowFloats, kPer = (kQuads * NR + kSoft - 1) / kSoft;
    constexpr int kChunk = 2 * S::kStages * NB * S::kBox / (4 * kSlot) < kSoft ? 2 * S::kStages * NB * S::kBox / (4 * kSlot) : kSoft;
    const int tid = threadIdx.x;
    float *ring = reinterpret_cast<float *>(&sm.k);
    float m[kPer], l[kPer];
    float4 x[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.f;
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int c0 = 0; c0 < parts; c0 += kChunk) {
        const int n = min(kChunk, parts - c0);
        fence_proxy_async();         // what the block wrote and read there before
        fence_proxy_async_global();  // the partials, written with plain stores
        named_bar_sync(1, kSoft);
        if (tid == 0) mbar_arrive_expect_tx(&sm.joined, uint32_t(n * kSlot * 4));
        named_bar_sync(1, kSoft);
        if (tid < n) {
            const int c = c0 + tid;
            bulk_load(ring + tid * kSlot, p0 + int64_t(c) * (2 * kSlot) + (c == 0 ? kSlot : 0), uint32_t(kSlot * 4), &sm.joined);
        }
        wait_warp(&sm.joined, round++ & 1, &sm.abort, 20000000);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int e = tid + k * kSoft, r = e / kQuads, d = 4 * (e % kQuads);
            if (r >= t.rows) break;
#pragma unroll 4
            for (int c = 0; c < n; ++c) {
                const float *row = ring + c * kSlot + r * S::kRowFloats;
                const float2 ml = *reinterpret_cast<const float2 *>(row + 128 * NB);
                const float4 v = *reinterpret_cast<const float4 *>(row + d);
                const float top = of_order(max(order_of(m[k]), order_of(ml.x)));
                const float f = weight_of(m[k], top), w = weight_of(ml.x, top);
                l[k] = f * l[k] + w * ml.y;
                x[k].x = f * x[k].x + w * v.x;
                x[k].y = f * x[k].y + w * v.y;
                x[k].z = f * x[k].z + w * v.z;
                x[k].w = f * x[k].w + w * v.w;
                m[k] = top;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int e = tid + k * kSoft, r = e / kQuads, d = 4 * (e % kQuads);
        if (r >= t.rows || d >= a.head_dim) continue;
        const float inv = inverse_of(l[k]);
        *reinterpret_cast<uint2 *>(out_row(a, t, r) + d) =
            make_uint2(act_t2<T>(x[k].x * inv, x[k].y * inv), act_t2<T>(x[k].z * inv, x[k].w * inv));
    }
}

__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

template <bool F8, bool BF16, int NB, int NR>
__device__ __forceinline__ void soft_role(const KvAttnArgs &a, Smem<NB, NR> &sm, Share<NR> share, uint32_t tbase, int total,
                                          int grid)
{
    using S = Shape<NB, NR>;
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    constexpr int kSlot = NR * S::kRowFloats;
    const int tid = threadIdx.x, lane = tid % 32, cta = blockIdx.x, u_end = share.u_end;
    Tile t, kept[2];
    bool kept_any[2] = {false, false};  // partials of a tile that began before, of one that ends behind
    uint32_t step = 0;
#pragma unroll 1
    while (share.next(t)) {
        place_rows<NB, NR>(a, sm, t);
        named_bar_sync(1, kSoft);
        if (steps_of(t)) {
            cut_queries<F8, BF16, NB, NR>(a, sm, t);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full);
            named_bar_sync(1, kSoft);  // the rows' scales are written
        }
        State<NB, NR> st;
        st.vref = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            st.m[r] = -INFINITY;
            st.l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < NB; ++c) st.o[c][r] = 0.f;
        }
        attend<F8, NB, NR>(a, sm, t, step, tbase, st);
        finish<T, NB, NR>(a, sm, t, st, t.whole ? nullptr : a.partials + int64_t(2 * cta + (t.first ? 1 : 0)) * kSlot);
        if (!t.whole) {
            if (t.first) kept[1] = t;
            else kept[0] = t;
            kept_any[t.first] = true;
        }
    }
    // Every partial of the block is written: it arrives at the counters of their tiles (of the
    // tile's first block), and joins the parts of those that it is the last to arrive at.
    if (!kept_any[0] && !kept_any[1]) return;
    if (tid == 0) {
        auto owner = [&](int x) {
            int c = min(grid - 1, int(float(x) * (float(grid) / float(total))));  // near the block that holds unit x
            while (c > 0 && kv_share(total, c, grid) > x) --c;
            while (kv_share(total, c + 1, grid) <= x) ++c;
            return c;
        };
        int c0[2], parts[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (kept_any[i]) {
                c0[i] = i ? cta : owner(kept[i].u0);
                parts[i] = (kept[i].u1 - 1 < u_end ? cta : owner(kept[i].u1 - 1)) - c0[i] + 1;
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
    named_bar_sync(1, kSoft);
    uint32_t round = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
        if (kept_any[i] && sm.parts[i])
            join_parts<T, NB, NR>(a, sm, i ? kept[1] : kept[0], a.partials + int64_t(sm.first[i]) * (2 * kSlot), sm.parts[i], round);
}

template <bool F8, bool BF16, int NB, int NR>
__device__ __forceinline__ void attend_rows(const CUtensorMap &km, const CUtensorMap &vm, const KvAttnArgs &a)
{
    using S = Shape<NB, NR>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t fin;
    Smem<NB, NR> &sm = *reinterpret_cast<Smem<NB, NR> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int *before = sm.before;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
            mbar_init(&sm.scales[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], kSoft / 32);
            mbar_init(&sm.o_full[i], 1);
        }
        mbar_init(&sm.q_full, kSoft / 32);
        mbar_init(&sm.joined, 1);
        mbar_init(&fin, 1);
        sm.abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    if (!a.behind_tiles) grid_dep_wait();  // queries, cache and batch arrays may come from the kernel before
    // Behind the wait: a kernel ahead that let its dependents start before it had its own Tensor Memory
    // would otherwise wait for columns that this block holds while it waits for that kernel.  (The tile
    // kernel of the same call holds its own by then.)
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&sm.tmem, S::kTmem);
        tc::tmem_relinquish();
    }

    // units of every sequence, summed up: each thread takes a run of sequences
    const bool split = a.partials != nullptr;
    const int per = (a.n_seqs + kThreads - 1) / kThreads;
    int shift = kUnitShift;
    auto units_of = [&](int b) {
        const int len = a.seq_len[b];
        const KvSpan s = kv_span(a.cu_q[b], a.cu_q[b + 1], len, a.M, a.capacity);
        if (len > a.capacity) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
        if (int64_t(s.n) * a.group > a.few_rows) return int64_t(0);
        return kv_tiles(s.n, a.group, NR) * a.kv_heads * (split ? kTileUnits + kv_units(s.len, shift) : 1);
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
        if (lane == 31) sm.units[warp] = sum;
        __syncthreads();
        all = 0;
        int64_t below = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) below += sm.units[w];
            all += sm.units[w];
        }
        sum += below - mine;
        if (all <= kMostUnits || shift == 30) break;
        __syncthreads();
    }
    // (still more: sequences that overlap, so that there are more rows than the call has; none is done)
    const int total = all <= kMostUnits ? int(all) : 0;
    if (tid == 0 && all > kMostUnits) atomicCAS(&g_kv_attn_error, kErrNone, kErrRange);
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < a.n_seqs) {
            before[b] = int(sum);
            sum += per > 1 ? units_of(b) : mine;
        }
    }
    if (tid == 0) before[a.n_seqs] = total;
    // no more shares than units, so that no block between a tile's first and last is without one
    const int least = split ? kTileUnits + kLeastUnits : 1;
    const int grid = min(int(gridDim.x), total / least + (total % least != 0)), cta = blockIdx.x;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    grid_dep_launch();  // (after the Tensor Memory is taken: the next kernel may want all of it)
    const uint32_t tbase = sm.tmem;
    if (cta >= grid) {
        if (warp == kMmaWarp) tc::tmem_dealloc(tbase, S::kTmem);
        return;
    }
    const Share<NR> share{a, before, shift, kv_share(total, cta, grid), kv_share(total, cta + 1, grid)};
    if (warp < kSoft / 32) {
        soft_role<F8, BF16, NB, NR>(a, sm, share, tbase, total, grid);
    } else if (warp == kCopyWarp) {
        copy_role<NB, NR>(a, &km, &vm, sm, share);
    } else if (lane == 0) {
        mma_role<F8, NB, NR>(a, sm, share, tbase, &fin);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tbase, S::kTmem);
}

template <bool F8, bool BF16, int NB, int NR>
__global__ void __launch_bounds__(kThreads, Shape<NB, NR>::kPerSm)
kv_attn_rows_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                    const __grid_constant__ KvAttnArgs a)
{
    attend_rows<F8, BF16, NB, NR>(km, vm, a);
    if (a.behind_tiles) grid_dep_wait();
}

struct RowsPlan {
    const void *fn;
    int per_sm;
    size_t smem;  // without the counts of `before`
};

template <bool F8, bool BF16, int NB, int NR>
RowsPlan rows_plan()
{
    using M = Smem<NB, NR>;
    constexpr size_t smem = offsetof(M, before) + 1024;
    static_assert(smem + (kKvMaxSeqs + 1) * sizeof(int) + sizeof(uint64_t) <= 232448, "a block's shared memory (and `fin`)");
    return {reinterpret_cast<const void *>(kv_attn_rows_kernel<F8, BF16, NB, NR>), Shape<NB, NR>::kPerSm, smem};
}

template <bool F8, bool BF16>
RowsPlan rows_plan(int head_dim)
{
    return head_dim <= 128 ? rows_plan<F8, BF16, 1, kRowsOfTile>() : rows_plan<F8, BF16, 2, kRowsOfTile>();
}

constexpr int kMostPerSm = 2;
// two partial slots a block in the workspace's 64 KB per SM: two blocks of 8 rows of 132 binary32
// values, or one of 8 rows of 260
static_assert(2 * 2 * kRowsOfTile * (128 + 4) * 4 <= 65536 && 2 * kRowsOfTile * (256 + 4) * 4 <= 65536, "");

}  // namespace

// Partials of two slots for every block, then the arrival counters (self-resetting).
size_t kv_attn_rows_workspace()
{
    return ws_scratch_bytes() + size_t(device_info().sm_count) * kMostPerSm * sizeof(unsigned);
}

// Keys and values as (page and head, slot, byte): bytes behind the head are not read, the copy
// fills zeros beyond the first dimension.
wq_status encode_cache(CUtensorMap *km, CUtensorMap *vm, const KvAttnArgs &a, int rows)
{
    const uint64_t dims[3] = {uint64_t(a.head_dim), uint64_t(1) << a.page_shift, uint64_t(a.num_pages) * a.kv_heads};
    const uint64_t strides[2] = {uint64_t(a.pitch), uint64_t(a.pitch) << a.page_shift};
    const uint32_t box[3] = {128, uint32_t(rows), 1};
    wq_status rc = encode_tmap(km, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.k, dims, strides, box, 128);
    return rc != WQ_OK ? rc : encode_tmap(vm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.v, dims, strides, box, 128);
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
    const RowsPlan p = f8 ? (bf16 ? rows_plan<true, true>(a.head_dim) : rows_plan<true, false>(a.head_dim))
                          : (bf16 ? rows_plan<false, true>(a.head_dim) : rows_plan<false, false>(a.head_dim));
    const size_t smem = p.smem + size_t(a.n_seqs + 1) * sizeof(int);
    if (cudaFuncSetAttribute(p.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(p.smem + (kKvMaxSeqs + 1) * sizeof(int))) != cudaSuccess)
        return check_launch("cudaFuncSetAttribute(kv_attn_rows_kernel)");
    CUtensorMap km, vm;
    wq_status rc = encode_cache(&km, &vm, a, std::min(1 << a.page_shift, kKeys));
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
    // Sequences with few rows per key head are bound by reading their keys once and go to the key-split
    // kernel, the others to the tile kernel.  One launch where the call's rows are so few that tiles would
    // leave most SMs idle, even if each key is read for several tiles of 8 rows, and for decode and draft
    // batches (kv_few_rows).
    // Tiles against split, us: heads of 128, 3000 keys, 1280 rows in all 80 / 37, 3200 rows 83 / 69,
    // 6400 rows 79 / 119; 64 rows and 20000 keys 382 / 22; heads of 256, 1280 rows 88 / 51, 3200 rows
    // 88 / 107.  Both kernels against the split alone, single tokens over 1000 keys and a chunk among
    // them, 32 query and key heads: 64 and 900 tokens 173 / 372, 200 and 2000 462 / 1110, 64 and 256 154 /
    // 208; 256 and 512 of 8 key heads 172 / 262.  What the tile kernel costs a draft batch, of which it
    // takes nothing: 64 sequences of 6 tokens 143.8 / 142.6, 512 of 2 960 / 950.
    const bool bf16 = dt == WQ_BF16, f8 = cache->format == WQ_FMT_E4M3;
    const int64_t idle = int64_t(a.head_dim <= 128 ? 24 : 16) * device_info().sm_count;
    a.few_rows = kv_few_rows(M, batch->n_seqs, q_heads, cache->kv_heads, idle);
    if (a.few_rows != 0x7fffffff) {
        rc = kv_attn_tiles(a, bf16, f8, stream);
        if (rc != WQ_OK) return rc;
        a.behind_tiles = true;
    }
    return kv_attn_rows(a, bf16, f8, stream);
}
