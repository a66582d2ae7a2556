// wq_kv_tiles.cu -- kv_attention for many rows per key head (prefill): 256 rows a block (128 for
// heads above 128) on the 5th-generation tensor cores (tcgen05).
//
// Mathematics (as in wq_kv_attn.cu): S = Q Kc^T per step of 128 (64) keys, x = S * (ks * sm_scale *
// log2 e), running maximum m and weight sum l in binary32, P = 2^(x - m) * vs / vref in binary16,
// O += P Vc, out = O * vref / l.  Codes are exact in binary16.  vref is a power of two above
// every value scale so far, so that P fits binary16 whatever the scales are.
//
// Bound by the tensor cores and by the 32 x 1024 exponentials of a 256 x 128 step, which cost
// about as much; so the two 128-row tiles of a block take turns: while one tile's products run,
// the other tile's softmax does (heads above 128: one tile, see Layout).
//  * warps 0-3 / 4-7: tile 0 / 1, a thread per row: query row to shared memory, then per step:
//    scores from Tensor Memory, weights back over them as the A operand of the second product.  O
//    stays in Tensor Memory; it is rescaled only when the maximum rose too far or a larger value
//    scale arrived, which is rare after the first steps.
//  * warps 8-11 (4-11): codes widened to binary16 into the 128-byte swizzled layout of the MMA's K-major
//    operands: keys as rows of dimensions, values transposed as rows of keys.
//  * warp 12: one thread issues the MMAs.
//  * warp 13: brings the next block's codes into shared memory (TMA) and its scales.
// Every wait is bounded; on expiry the block records an error, stops and frees its Tensor Memory.
//
// Measured (device time, calls back to back in a graph): two chunks of 2048 tokens, 32 query and 8 key
// heads of 128, behind 4096 to 6000 keys: 540 us, 768 TF/s.  Four of 1000 tokens behind 2000 keys, heads
// of 256: 550 us, 596 TF/s (3843 us by the split kernel of wq_kv_attn.cu).  Five prompts of 100 to 1100
// tokens, 32 heads: 70 us (84 us by a caller's clock), where a block's start and end are most of its 18
// to 25 us.  While it was built: codes by TMA instead of by the widening warps'
// own loads: 1050 -> 678 us for the chunks; weights in one pass where the references hold: 678 ->
// 641; loops of the roles rolled, so that their code stays in the instruction cache: 93 -> 87 us for
// the prompts.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "wq_act.cuh"
#include "wq_kv_attn.cuh"
#include "wq_tc.cuh"

namespace wq {

static __device__ int g_kv_tiles_error;

int kv_tiles_read_error()
{
    int v = 0, zero = 0;
    cudaMemcpyFromSymbol(&v, g_kv_tiles_error, sizeof v);
    cudaMemcpyToSymbol(g_kv_tiles_error, &zero, sizeof zero);
    return v;
}

namespace {

constexpr int kTile = 128;           // rows of a tile: MMA M
constexpr int kMaxGroups = 8;        // groups of 16 keys of a step (a group lies in one page)
constexpr int kMmaWarp = 12, kCopyWarp = 13;  // (14 warps leave 128 registers a thread)
constexpr int kThreads = 32 * (kCopyWarp + 1);
__device__ __forceinline__ float log2_approx(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t x, y, z, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    memcpy(&z, &c, 8);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    memcpy(&a, &d, 8);
    return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    memcpy(&a, &d, 8);
    return a;
}

constexpr int kRing = 4;             // scale sets: a set is rewritten once both tiles are two steps on
constexpr uint32_t kTmemCols = 512, kScol = 0, kOcol = 256;  // two 128-column tiles of each

// Value scales that may be part of the weights' exponent (weights_once): the least is 2^-81 of the
// reference above the largest, so that a weight vanishes only under 2^-55 and a group's sum over its
// scale stays within binary32.
constexpr float kLeastPlain = 0x1p-48f, kMostPlain = 0x1p32f;

// Up to here weights_once takes a row's maximum: it and the shifts are one binary32 number there, off by
// half a step of it (2^-4; from 2^26 on weights would not fit binary16).
constexpr float kWide = 0x1p20f;

// Weights are raised by 2^kRaise: exact to half a step down to 2^-(14 + kRaise) in binary16.  A
// maximum that rises a little is not followed while all weights fit: 2^kRaise times the rise.
constexpr float kRaise = 11.f;

struct Bars {
    uint64_t q_full, k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_done[2], sc_full[kRing];
    uint64_t raw_k_full, raw_k_free, raw_v_full, raw_v_free, fin;
};
struct Scales {
    float k[kRing][kMaxGroups];    // key scale * |sm_scale| * log2 e
    float v[kRing][kMaxGroups];    // value scale, its logarithm and inverse
    float log_v[kRing][kMaxGroups], inv_v[kRing][kMaxGroups];
    float v_max[kRing];
    uint32_t dead[kRing];          // groups whose block-table entry is no page
    int plain[kRing];              // no dead groups, all value scales in kLeastPlain .. kMostPlain
};

// DT: the head's size rounded up to 64, 128 or 256.  Up to 128: two tiles of 128 rows, steps of 128
// keys.  256: the sums of one tile take half of the Tensor Memory and two steps of 128 keys do not fit
// shared memory, so one tile in steps of 64 keys, with scores of two steps in Tensor Memory so that
// products and softmax still overlap; the second tile's warps widen codes instead.
template <int DT>
struct Layout {
    static constexpr bool kTwo = DT <= 128;
    static constexpr int kRows = kTwo ? 2 * kTile : kTile;  // of a block
    static constexpr int kKeys = kTwo ? 128 : 64;           // of a step
    static constexpr int kGroups = kKeys / 16;
    static constexpr int kSoftWarps = kTwo ? 8 : 4, kConvWarps = kMmaWarp - kSoftWarps;
    static constexpr int kBoxes = DT <= 128 ? 1 : 2;        // boxes of 128 bytes of a key
    static constexpr int kAtom = kTile * 128;               // 128 query rows of 64 binary16
    static constexpr int kQ = DT / 64 * kAtom;              // a query tile
    static constexpr int kKAtom = kKeys * 128;              // the same of a step's keys
    static constexpr int kK = DT / 64 * kKAtom;
    static constexpr int kV = 2 * DT * kKeys;               // DT rows of keys
    static constexpr int kRaw = kKeys * 128 * kBoxes;       // codes of a step
    static constexpr int kBytes = kRows / kTile * kQ + 2 * kK + 2 * kV + 2 * kRaw;
    // the scores of (tile, step): their columns, and the parity of their barriers
    static constexpr uint32_t kSCols = kTwo ? 128 : 64;
    __device__ static __forceinline__ int slot(int tile, int j) { return kTwo ? tile : j & 1; }
    __device__ static __forceinline__ uint32_t parity(int j) { return (kTwo ? j : j >> 1) & 1; }
};

__device__ __forceinline__ uint64_t globaltimer()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits at most about 2 s, or 20 ms once another role gave up.  wait_warp: the whole warp, with one
// answer, so that a warp gives up together.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait_short(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_short(bar, parity)) return true;
        if (globaltimer() - t0 > (*abort ? 20000000ull : 2000000000ull)) {
            atomicCAS(&g_kv_tiles_error, kErrNone, kErrWaitTimeout);
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

struct Item {
    KvSpan s;
    int b, head, row0, rows;  // the block's rows
    int keys;                 // keys that its last row sees
    int steps, tiles;         // key steps of the block (of its last tile)
    int steps_of[2];          // of each tile: the first sees fewer keys
};

// ------------------------------------------------------------------ codes to shared memory
// A step's codes arrive as boxes per page part of 128 bytes a key (zeros behind the head), in the
// 128-byte swizzle; lanes look up a page each, of a box or of a group and its scales.
template <int DT>
__device__ __forceinline__ void copy_role(const KvAttnArgs &a, const Item &t, const CUtensorMap *km, const CUtensorMap *vm,
                                          uint8_t *kraw, uint8_t *vraw, Scales &sc, Bars &bar, volatile int *abort)
{
    constexpr int kKeys = Layout<DT>::kKeys, kGroups = Layout<DT>::kGroups, kBoxes = Layout<DT>::kBoxes;
    const int lane = threadIdx.x % 32;
    const int32_t *table = a.block_table + int64_t(t.b) * a.max_pages;
    const int box_rows = min(1 << a.page_shift, kKeys), boxes = kKeys / box_rows;
    // lane l: the page of box l, lane kGroups + l: that of group l
    const int my_key = lane < kGroups ? lane * box_rows : (lane - kGroups) * 16;
    const bool boxed = lane < boxes, grouped = lane >= kGroups && lane < 2 * kGroups;
    auto entry_of = [&](int step) {
        const int key = step * kKeys + my_key;
        return (boxed || grouped) && key < t.keys ? table[key >> a.page_shift] : 0;
    };
    int entry = entry_of(0), sent_k = 0, sent_v = 0;
    for (int j = 0; j < t.steps; ++j) {
        const int key = j * kKeys + my_key;
        const bool used = (boxed || grouped) && key < t.keys;
        const int64_t page = used ? kv_page_ok(entry, a.num_pages) : -1;
        const int z = page < 0 ? -1 : int(page) * a.kv_heads + t.head;
        float ks = 0.f, vs = 0.f;
        if (grouped && z >= 0) {
            ks = a.k_scale[z];
            vs = a.v_scale[z];
        }
        if (j + 1 < t.steps) entry = entry_of(j + 1);
        const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, boxed && z >= 0))) * uint32_t(box_rows * 128 * kBoxes);
        const int y = key & ((1 << a.page_shift) - 1);
        if (j && !wait_warp(&bar.raw_k_free, (j - 1) & 1, abort)) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.raw_k_full, bytes);
        __syncwarp();
        if (boxed && z >= 0)
#pragma unroll
            for (int c = 0; c < kBoxes; ++c)
                tma_load_3d(kraw + c * kKeys * 128 + lane * box_rows * 128, km, 128 * c, y, z, &bar.raw_k_full);
        sent_k = j + 1;
        if (j && !wait_warp(&bar.raw_v_free, (j - 1) & 1, abort)) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar.raw_v_full, bytes);
        __syncwarp();
        if (boxed && z >= 0)
#pragma unroll
            for (int c = 0; c < kBoxes; ++c)
                tma_load_3d(vraw + c * kKeys * 128 + lane * box_rows * 128, vm, 128 * c, y, z, &bar.raw_v_full);
        sent_v = j + 1;
        // ---- scales
        const int set = j % kRing, g = lane - kGroups;
        const bool bad = grouped && used && z < 0;
        const uint32_t dead = __ballot_sync(0xffffffffu, bad) >> kGroups;
        const bool normal = vs >= kLeastPlain && vs <= kMostPlain;
        // (groups behind the last key: masked by their keys, any scale will do)
        const bool plain = __all_sync(0xffffffffu, !grouped || !used || normal) && !dead;
        const float top = __uint_as_float(warp_umax(__float_as_uint(fabsf(vs))));
        if (grouped) {
            sc.k[set][g] = ks * fabsf(a.sm_scale) * kLog2e;
            sc.v[set][g] = vs;
            sc.log_v[set][g] = used ? log2_approx(vs) : 0.f;  // (all keys of an unused group are masked)
            sc.inv_v[set][g] = used ? 1.f / vs : 0.f;
        }
        if (lane == 0) {
            sc.dead[set] = dead;
            sc.plain[set] = plain;
            sc.v_max[set] = top;
            if (dead) atomicCAS(&g_kv_tiles_error, kErrNone, kErrRange);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.sc_full[set]);
    }
    // nothing may land in shared memory after the block exits
    if (sent_k) wait_warp(&bar.raw_k_full, (sent_k - 1) & 1, abort);
    if (sent_v) wait_warp(&bar.raw_v_full, (sent_v - 1) & 1, abort);
}

// ------------------------------------------------------------------ codes to binary16
template <bool F8, int DT>
__device__ __noinline__ void convert_role(const KvAttnArgs &a, const Item &t, const uint8_t *kraw, const uint8_t *vraw, uint8_t *ksm,
                             uint8_t *vsm, const Scales &sc, Bars &bar, volatile int *abort)
{
    using L = Layout<DT>;
    constexpr int kKeys = L::kKeys;
    constexpr int kPerRow = DT / 16;                        // 16-byte chunks of a key
    constexpr int kPass = 32 * L::kConvWarps / kPerRow;     // keys of a pass
    constexpr int kKp = kKeys / kPass;                      // passes: 8 (DT 128) or 4
    constexpr int kKeyWarps = kKeys / 32, kDimWarps = L::kConvWarps / kKeyWarps;
    constexpr int kVt = DT / 32 / kDimWarps;                // value tasks (8 keys x 4 dimensions) of a thread
    const int ct = threadIdx.x - 32 * L::kSoftWarps, cw = ct / 32, lane = ct % 32;
    const int chunk = ct % kPerRow, krow = ct / kPerRow;
    // values: a warp takes 32 keys; its lanes 8 keys x 4 dimensions each, so that the transposed
    // 16-byte stores are free of conflicts
    const int tg = lane % 8 / 2, dg = 2 * (lane / 8) + lane % 2, vkey = 32 * (cw % kKeyWarps) + 8 * tg;
    for (int j = 0; j < t.steps; ++j) {
        const int buf = j & 1;
        uint8_t *kb = ksm + buf * Layout<DT>::kK, *vb = vsm + buf * Layout<DT>::kV;
        // ---- keys
        if (!wait_warp(&bar.raw_k_full, j & 1, abort)) return;
        if (j >= 2 && !wait_warp(&bar.k_free[buf], ((j >> 1) - 1) & 1, abort)) return;
#pragma unroll 1
        for (int i = 0; i < kKp; ++i) {
            const int r = krow + kPass * i;
            const uint4 raw = lds128(kraw + chunk / 8 * (kKeys * 128) + r * 128 + (((chunk % 8) ^ (r & 7)) << 4));
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            if constexpr (!F8) {
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] ^= 0x80808080u;
            }
            uint8_t *row = kb + chunk / 4 * Layout<DT>::kKAtom + r * 128;
            const uint4 lo = make_uint4(widen<F8, 0>(w[0]), widen<F8, 1>(w[0]), widen<F8, 0>(w[1]), widen<F8, 1>(w[1]));
            const uint4 hi = make_uint4(widen<F8, 0>(w[2]), widen<F8, 1>(w[2]), widen<F8, 0>(w[3]), widen<F8, 1>(w[3]));
            const int c = 2 * (chunk % 4);
            // the lanes of every other 64 dimensions store their halves in the other order: the atoms
            // share banks
            const bool swap = chunk / 4 % 2;
            sts128(row + (((c + swap) ^ (r & 7)) << 4), swap ? hi : lo);
            sts128(row + (((c + !swap) ^ (r & 7)) << 4), swap ? lo : hi);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.raw_k_free);
            mbar_arrive(&bar.k_full[buf]);
        }
        // ---- values
        if (!wait_warp(&bar.raw_v_full, j & 1, abort)) return;
        if (j >= 2 && !wait_warp(&bar.v_free[buf], ((j >> 1) - 1) & 1, abort)) return;
        int left = t.keys - j * kKeys - vkey;  // keys of the lane's eight that hold codes
        // a page that is none was not copied (its weights are 0, but e4m3 may hold NaN codes)
        if (F8 && wait_warp(&bar.sc_full[j % kRing], (j / kRing) & 1, abort) && (sc.dead[j % kRing] >> (vkey / 16) & 1)) left = 0;
#pragma unroll 1
        for (int i = 0; i < kVt; ++i) {
            const int d = cw / kKeyWarps * (DT / kDimWarps) + 32 * i + 4 * dg;
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = lds32(vraw + d / 128 * (kKeys * 128) + (vkey + e) * 128 + (((d % 128 / 16) ^ e) << 4) + (d & 15));
            if (F8 && left < 8) {
                // slots behind the last key hold anything, e4m3 NaN codes among it
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= left) w[e] = 0u;
            }
            uint32_t o[4][4];  // [dimension][pair of keys]
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t x = prmt(w[2 * e], w[2 * e + 1], 0x5140);
                uint32_t y = prmt(w[2 * e], w[2 * e + 1], 0x7362);
                if constexpr (!F8) {
                    x ^= 0x80808080u;
                    y ^= 0x80808080u;
                }
                o[0][e] = widen<F8, 0>(x);
                o[1][e] = widen<F8, 1>(x);
                o[2][e] = widen<F8, 0>(y);
                o[3][e] = widen<F8, 1>(y);
            }
            uint8_t *base = vb + vkey / 64 * (DT * 128);
            const int c = vkey % 64 / 8;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                sts128(base + (d + x) * 128 + ((c ^ ((d + x) & 7)) << 4), make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&bar.raw_v_free);
            mbar_arrive(&bar.v_full[buf]);
        }
    }
}

// ------------------------------------------------------------------ MMA issue (one thread)
template <int DT>
__device__ void mma_role(const KvAttnArgs &a, const Item &t, uint32_t qaddr, uint32_t kaddr, uint32_t vaddr, Bars &bar,
                         uint32_t tbase, volatile int *abort)
{
    using L = Layout<DT>;
    const uint32_t iqk = tc::idesc_f16(false, kTile, L::kKeys), ipv = tc::idesc_f16(false, kTile, DT);
    // descriptors differ in their address field only: the offsets below are constants added to the
    // low word
    const uint64_t dq = tc::sdesc_sw128(qaddr), dk = tc::sdesc_sw128(kaddr), dv = tc::sdesc_sw128(vaddr);
    const uint32_t high = uint32_t(dq >> 32), q_lo = uint32_t(dq), k_lo = uint32_t(dk), v_lo = uint32_t(dv);
    auto desc = [&](uint32_t lo) { return uint64_t(high) << 32 | lo; };
    auto qk = [&](int tile, int j) {
        const uint32_t q = q_lo + uint32_t(tile * L::kQ >> 4), k = k_lo + uint32_t((j & 1) * L::kK >> 4);
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) {
            const uint32_t at = uint32_t(i & 3) * 32;
            tc::mma_f16_ss(tbase + kScol + L::kSCols * L::slot(tile, j), desc(q + (((i >> 2) * L::kAtom + at) >> 4)),
                           desc(k + (((i >> 2) * L::kKAtom + at) >> 4)), iqk, i > 0);
        }
        tc::commit(&bar.s_full[L::slot(tile, j)]);
    };
    auto pv = [&](int tile, int j) {
        const uint32_t v = v_lo + uint32_t((j & 1) * L::kV >> 4);
#pragma unroll
        for (int i = 0; i < L::kGroups; ++i) {
            const uint32_t off = uint32_t(((i >> 2) * (DT * 128) + (i & 3) * 32) >> 4);
            tc::mma_f16_ts(tbase + kOcol + 128 * tile, tbase + kScol + L::kSCols * L::slot(tile, j) + 8 * i, desc(v + off), ipv,
                           j > 0 || i > 0);
        }
        tc::commit(&bar.o_done[tile]);
    };
    if (!wait(&bar.q_full, 0, abort) || !wait(&bar.k_full[0], 0, abort)) return;
    tc::fence_after_sync();
    for (int tile = 0; tile < t.tiles; ++tile)
        if (t.steps_of[tile]) qk(tile, 0);
    tc::commit(&bar.k_free[0]);
    bool ok = true;
    if constexpr (!L::kTwo) {
        // the next step's scores go over the weights of the step before, whose product is in the pipe
        for (int j = 0; j < t.steps; ++j) {
            if (j + 1 < t.steps) {
                if (!wait(&bar.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, abort)) break;
                tc::fence_after_sync();
                qk(0, j + 1);
                tc::commit(&bar.k_free[(j + 1) & 1]);
            }
            if (!wait(&bar.p_full[j & 1], L::parity(j), abort) || !wait(&bar.v_full[j & 1], (j >> 1) & 1, abort)) break;
            tc::fence_after_sync();
            pv(0, j);
            tc::commit(&bar.v_free[j & 1]);
        }
        ok = false;
    }
    for (int j = 0; j < t.steps && ok; ++j) {
        const int buf = j & 1, nbuf = buf ^ 1;
        bool have_v = false, have_k = false;
        for (int tile = 0; tile < t.tiles; ++tile) {
            if (j >= t.steps_of[tile]) continue;
            ok = wait(&bar.p_full[tile], j & 1, abort) && (have_v || wait(&bar.v_full[buf], (j >> 1) & 1, abort));
            if (!ok) break;
            have_v = true;
            tc::fence_after_sync();
            pv(tile, j);
            if (j + 1 < t.steps_of[tile]) {
                if (!have_k) {
                    ok = wait(&bar.k_full[nbuf], ((j + 1) >> 1) & 1, abort);
                    if (!ok) break;
                    have_k = true;
                    tc::fence_after_sync();
                }
                qk(tile, j + 1);  // behind the tile's second product in the pipe: it may overwrite the weights
            }
        }
        if (!ok) break;
        tc::commit(&bar.v_free[buf]);
        if (j + 1 < t.steps) tc::commit(&bar.k_free[nbuf]);
    }
    tc::commit(&bar.fin);  // all MMAs complete before the Tensor Memory is freed
    wait(&bar.fin, 0, abort);
}

// ------------------------------------------------------------------ softmax (a thread per row)
// The weights of a step in one pass over its scores (see softmax_role), stored over them if all of
// the warp fit binary16 (true; any: whatever they are), else nothing is.  MASKED: some row sees fewer
// than all keys.
template <bool MASKED, int GROUPS>
__device__ __forceinline__ bool weights_once(uint32_t scol, const float *ks, const float *log_v, const float *inv_v,
                                             float unscale, float shift, int left, float &lsum, bool any)
{
    uint32_t p[GROUPS / 2][16], s[2][16];
    float most = 0.f;
    tc::ld_32x32b_x16(scol, s[0]);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        tc::wait_ld();
        if (g + 1 < GROUPS) tc::ld_32x32b_x16(scol + 16 * (g + 1), s[(g + 1) & 1]);
        if (MASKED)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * g + i >= left) s[g & 1][i] = 0xff800000u;  // -inf: weight 0
        // (a scale of 0 times -inf would be NaN)
        const float k = MASKED ? fmaxf(ks[g] * unscale, 0x1p-126f) : ks[g] * unscale, off = log_v[g] + shift;
        const float2 k2 = make_float2(k, k), off2 = make_float2(off, off);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float2 e = fma2(make_float2(__uint_as_float(s[g & 1][i]), __uint_as_float(s[g & 1][i + 1])), k2, off2);
            const float2 w = make_float2(exp2_approx(e.x), exp2_approx(e.y));
            sum = add2(sum, w);
            p[g / 2][8 * (g % 2) + i / 2] = act_t2<__half>(w.x, w.y);
        }
        const float both = sum.x + sum.y;
        most = both <= 61440.f ? most : INFINITY;  // (NaN too)
        lsum = fmaf(both, inv_v[g], lsum);
    }
    if (!__all_sync(0xffffffffu, most == 0.f || any)) return false;
#pragma unroll
    for (int c = 0; c < GROUPS / 2; ++c) tc::st_32x32b_x16(scol + 16 * c, p[c]);
    tc::wait_st();
    return true;
}

// The running references after a step: the maximum m over its scores too and, vref, a power of two
// above its value scales, with l and the output tile taken over to them.  False: gave up.
// (Loops over chunks of 32 keys stay loops: unrolled, the roles' code does not fit the instruction
// cache, and blocks of few steps run it cold.)
template <int DT>
__device__ __forceinline__ bool new_references(uint32_t scol, uint32_t ocol, const Scales &sc, int set, float unscale,
                                               int left, bool all, uint32_t dead, int j, int tile, Bars &bar,
                                               volatile int *abort, float &m, float &vref, float &l)
{
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < Layout<DT>::kGroups / 2; ++c) {
        uint32_t s[32];
        tc::ld_32x32b_x32(scol + 32 * c, s);
        tc::wait_ld();
        if (!all) {
#pragma unroll
            for (int x = 0; x < 32; ++x)
                if (32 * c + x >= left || (dead >> (2 * c + x / 16) & 1)) s[x] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y[4];  // (scales are not negative: the largest product is the largest score's)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                y[x] = fmaxf(__uint_as_float(s[16 * h + x]), __uint_as_float(s[16 * h + 4 + x]));
                y[x] = fmaxf(fmaxf(y[x], __uint_as_float(s[16 * h + 8 + x])), __uint_as_float(s[16 * h + 12 + x]));
            }
            const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            // -inf stays -inf where a scale is 0
            mx = fmaxf(mx, top == -INFINITY ? top : top * (sc.k[set][2 * c + h] * unscale));
        }
    }
    const float m_new = fmaxf(m, mx), vmax = sc.v_max[set];
    const float vnew = vmax >= vref && vmax > 0.f ? __uint_as_float((__float_as_uint(vmax) & 0x7f800000u) + 0x00800000u) : vref;
    const float fm = m_new == m ? 1.f : exp2_approx(m - m_new);
    const float fo = vnew == vref ? fm : fm * (vref * (1.f / vnew));
    l *= fm;
    m = m_new;
    vref = vnew;
    if (j > 0 && __any_sync(0xffffffffu, fo != 1.f)) {
        if (!wait_warp(&bar.o_done[tile], (j - 1) & 1, abort)) return false;
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < DT / 32; ++c) {
            uint32_t o[32];
            tc::ld_32x32b_x32(ocol + 32 * c, o);
            tc::wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fo);
            tc::st_32x32b_x32(ocol + 32 * c, o);
        }
        tc::wait_st();
    }
    return true;
}

// The weights of a step with groups that are no pages, or with value scales or a maximum that weights_once
// does not take, after new_references: no score is over the maximum.
template <int GROUPS>
__device__ __forceinline__ void weights_any(uint32_t scol, const Scales &sc, int set, float unscale, int left, uint32_t dead,
                                            float m, float vref, float &l)
{
    const float top = m == -INFINITY ? 0.f : m, inv = vref > 0.f ? 1.f / vref : 0.f;
#pragma unroll 1
    for (int g = 0; g < GROUPS; ++g) {
        uint32_t s[16], p[8];
        tc::ld_32x32b_x16(scol + 16 * g, s);
        tc::wait_ld();
        const float k = sc.k[set][g] * unscale, v = sc.v[set][g] * inv;
        const bool gone = dead >> g & 1;
#pragma unroll
        for (int x = 0; x < 16; x += 2) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // (the product as new_references rounds it: never over the maximum)
                w[e] = exp2_approx(__fmul_rn(__uint_as_float(s[x + e]), k) - top + kRaise);
                if (16 * g + x + e >= left || gone) w[e] = 0.f;
            }
            l += w[0] + w[1];
            p[x / 2] = act_t2<__half>(w[0] * v, w[1] * v);
        }
        tc::st_32x32b_x8(scol + 8 * g, p);
    }
    tc::wait_st();
}

template <bool BF16, int DT>
__device__ void softmax_role(const KvAttnArgs &a, const Item &t, uint8_t *qsm, const Scales &sc, Bars &bar,
                             uint32_t tbase, volatile int *abort)
{
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    using L = Layout<DT>;
    constexpr int kKeys = L::kKeys, kGroups = L::kGroups, kBoxes = L::kBoxes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, tile = warp / 4;
    if (tile >= t.tiles) return;
    const int r = 32 * (warp % 4) + lane, row = tile * kTile + r;
    const bool live = row < t.rows;
    const int i = live ? (t.row0 + row) / a.group : 0, h = live ? (t.row0 + row) % a.group : 0;
    const int64_t at = (int64_t(t.s.q0 + i) * a.q_heads + t.head * a.group + h) * a.head_dim;
    const int seen = live ? t.s.len - t.s.n + i + 1 : 0;
    const uint32_t tlane = tbase + (uint32_t(32 * (warp % 4)) << 16);
    const uint32_t ocol = tlane + kOcol + 128 * tile;

    // ---- the warp's 32 query rows to shared memory, a row at a time across the lanes: with
    // sm_scale's sign, binary16 (bfloat16 rows scaled by a power of two so that the largest value
    // fits: what is lost below is under 2^-25 of it)
    const int steps = t.steps_of[tile];
    const uint32_t lives = __ballot_sync(0xffffffffu, live);
    const int d4 = 4 * lane;  // the lane's four values of a row (or of each of its halves)
    uint8_t *rows_sm = qsm + tile * Layout<DT>::kQ + 32 * (warp % 4) * 128;
    float unscale = 1.f;
    constexpr int kBatch = 8 / kBoxes;  // rows whose loads are in flight together
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += kBatch) {
        uint2 x[kBatch][kBoxes];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t from = __shfl_sync(0xffffffffu, at, r0 + k);
#pragma unroll
            for (int c = 0; c < kBoxes; ++c)
                x[k][c] = (lives >> (r0 + k) & 1) && d4 + 128 * c < a.head_dim
                              ? *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + from + d4 + 128 * c)
                              : make_uint2(0, 0);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if constexpr (BF16) {
                float amax = 0.f;
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) {
                    const float2 lo = act_f2<T>(x[k][c].x), hi = act_f2<T>(x[k][c].y);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(lo.x), fabsf(lo.y)), fmaxf(fabsf(hi.x), fabsf(hi.y))));
                }
                amax = __uint_as_float(warp_umax(__float_as_uint(amax)));
                const int e = kv_clamp(int(__float_as_uint(amax) >> 23) - 127, -120, 120);
                const float up = copysignf(__uint_as_float(uint32_t(127 - e) << 23), a.sm_scale);
                if (lane == r0 + k) unscale = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) {
                    const float2 lo = act_f2<T>(x[k][c].x), hi = act_f2<T>(x[k][c].y);
                    x[k][c] = make_uint2(act_t2<__half>(lo.x * up, lo.y * up), act_t2<__half>(hi.x * up, hi.y * up));
                }
            } else if (a.sm_scale < 0.f) {
#pragma unroll
                for (int c = 0; c < kBoxes; ++c) {
                    x[k][c].x ^= 0x80008000u;
                    x[k][c].y ^= 0x80008000u;
                }
            }
#pragma unroll
            for (int c = 0; c < kBoxes; ++c) {
                const int d = d4 + 128 * c;
                if (d < DT)
                    *reinterpret_cast<uint2 *>(rows_sm + d / 64 * L::kAtom + (r0 + k) * 128 +
                                               (((d % 64 / 8) ^ ((r0 + k) & 7)) << 4) + d % 8 * 2) = x[k][c];
            }
        }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.q_full);

    float m = -INFINITY, l = 0.f, vref = 0.f;
    for (int j = 0; j < steps; ++j) {
        const int set = j % kRing, key0 = j * kKeys;
        const uint32_t scol = tlane + kScol + L::kSCols * L::slot(tile, j);
        if (!wait_warp(&bar.sc_full[set], (j / kRing) & 1, abort) ||
            !wait_warp(&bar.s_full[L::slot(tile, j)], L::parity(j), abort)) return;
        tc::fence_after_sync();
        const int left = seen - key0;  // keys of this step that the row sees
        const int least = __reduce_min_sync(0xffffffffu, left);
        // ---- One pass where the running references hold: no score too far over the maximum so far
        // shows as no group of weights summing up to more than binary16 holds (weights under the
        // maximum sum up to at most 16 * 2^kRaise = 2^15), so the sums that l needs anyway are the
        // check.  The weights stay in registers until it passed.  The value scale is part of the
        // exponent, P = 2^(x - m + kRaise + log2(vs / vref)), and l takes a group's sum back over
        // vs / vref.
        const uint32_t dead = sc.dead[set];
        const bool all_seen = least >= kKeys, plain = sc.plain[set];
        bool refer = j == 0 || !plain || !__all_sync(0xffffffffu, sc.v_max[set] < vref && (fabsf(m) <= kWide || left <= 0));
#pragma unroll 1
        for (;;) {
            if (refer) {
                if (!new_references<DT>(scol, ocol, sc, set, unscale, left, all_seen && !dead, dead, j, tile, bar, abort, m, vref, l))
                    return;
                if (!plain || __any_sync(0xffffffffu, fabsf(m) > kWide && left > 0)) {
                    weights_any<kGroups>(scol, sc, set, unscale, left, dead, m, vref, l);
                    break;
                }
            }
            const float shift = kRaise - (m == -INFINITY ? 0.f : m) - float(int(__float_as_uint(vref) >> 23) - 127);
            float lsum = 0.f;
            const bool fits = all_seen
                                  ? weights_once<false, kGroups>(scol, sc.k[set], sc.log_v[set], sc.inv_v[set], unscale, shift, left, lsum, refer)
                                  : weights_once<true, kGroups>(scol, sc.k[set], sc.log_v[set], sc.inv_v[set], unscale, shift, left, lsum, refer);
            if (fits) {
                l = fmaf(lsum, vref, l);
                break;
            }
            refer = true;
        }
        // One tile: the sums of the step before need not be done yet.  They run before this step's anyway;
        // waited for here, the barrier is never two phases behind a wait.
        if (!L::kTwo && j > 0 && !wait_warp(&bar.o_done[tile], (j - 1) & 1, abort)) return;
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[L::slot(tile, j)]);
    }
    if (steps > 0 && !wait_warp(&bar.o_done[tile], (steps - 1) & 1, abort)) return;
    tc::fence_after_sync();
    // ---- the finished rows: through the warp's part of the query rows' memory (its products are
    // done), so that rows leave as whole lines
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);  // (vref / l may be below the normal numbers)
    const uint32_t keep = l == 0.f ? 0u : ~0u;
    uint8_t *back = qsm + tile * Layout<DT>::kQ + 32 * (warp % 4) * (2 * DT);
    if (steps == 0) named_bar_sync(1 + tile, kTile);  // (no product said that all query rows are written)
#pragma unroll 1
    for (int c = 0; c < DT / 32; ++c) {
        uint32_t o[32];
        if (steps > 0) {
            tc::ld_32x32b_x32(ocol + 32 * c, o);
            tc::wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __uint_as_float(o[8 * k + 2 * e]) * inv * vref, y = __uint_as_float(o[8 * k + 2 * e + 1]) * inv * vref;
                h[e] = act_t2<T>(x, y) & keep;
            }
            sts128(back + lane * (2 * DT) + (((4 * c + k) ^ (lane & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
        }
    }
    __syncwarp();
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
        const int64_t to = __shfl_sync(0xffffffffu, at, k);
#pragma unroll
        for (int c = 0; c < kBoxes; ++c) {
            const int d = d4 + 128 * c;
            if ((lives >> k & 1) && d < a.head_dim)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to + d) =
                    lds64(back + k * (2 * DT) + (((d / 8) ^ (k & 7)) << 4) + d % 8 * 2);
        }
    }
}

template <bool F8, bool BF16, int DT>
__global__ void __launch_bounds__(kThreads, 1)
kv_attn_tiles_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                     const __grid_constant__ KvAttnArgs a)
{
    using L = Layout<DT>;
    constexpr int kRows = L::kRows, kKeys = L::kKeys;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Bars bar;
    __shared__ Scales sc;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, s_seq[6];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qsm = smem, *ksm = qsm + kRows / kTile * L::kQ, *vsm = ksm + 2 * L::kK;
    uint8_t *kraw = vsm + 2 * L::kV, *vraw = kraw + L::kRaw;
    volatile int *abort = &abort_flag;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    grid_dep_wait();  // queries, cache and batch arrays may come from the kernel before

    const int64_t item = blockIdx.x / a.kv_heads;
    if (tid == 0) {
        s_seq[0] = -1;
        s_seq[5] = 0;
        abort_flag = 0;
    }
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1], len = a.seq_len[b];
        const bool some = lo < hi;  // (slots without tokens may have any offsets)
        // a sequence that begins before the end of the last: no item's owner is certain, so nothing is done
        if (some && a.cu_q[max(b - 1, 0)] > lo) s_seq[5] = 1;
        const KvSpan s = kv_span(lo, hi, len, a.M, a.capacity);
        const int64_t first = kv_row_item(s.q0, b, a.group, kRows, a.by_rows);
        if (some && first <= item && item < kv_row_item(s.q0 + s.n, b + 1, a.group, kRows, a.by_rows)) {
            s_seq[0] = b;
            s_seq[1] = lo;
            s_seq[2] = hi;
            s_seq[3] = len;
            s_seq[4] = int(item - first);
        }
    }
    __syncthreads();
    Item t;
    t.b = s_seq[0];
    if (s_seq[5] && tid == 0) atomicCAS(&g_kv_tiles_error, kErrNone, kErrRange);
    if (t.b < 0 || s_seq[5]) return;
    t.s = kv_span(s_seq[1], s_seq[2], s_seq[3], a.M, a.capacity);
    if (tid == 0 && s_seq[3] > a.capacity) atomicCAS(&g_kv_tiles_error, kErrNone, kErrRange);
    const int all = t.s.n * a.group;
    // the last rows first: they see the most keys
    const int64_t k = kv_tiles(t.s.n, a.group, kRows) - 1 - s_seq[4];
    if (k < 0 || all <= a.few_rows) return;
    t.head = blockIdx.x % a.kv_heads;
    t.row0 = int(k) * kRows;
    t.rows = min(kRows, all - t.row0);
    t.keys = max(0, t.s.len - t.s.n + (t.row0 + t.rows - 1) / a.group + 1);
    t.steps = (t.keys + kKeys - 1) / kKeys;
    t.tiles = t.rows > kTile ? 2 : 1;
    const int first_keys = max(0, t.s.len - t.s.n + (t.row0 + min(t.rows, kTile) - 1) / a.group + 1);
    t.steps_of[0] = (first_keys + kKeys - 1) / kKeys;
    t.steps_of[1] = t.steps;

    if (tid == 0) {
        mbar_init(&bar.q_full, 4 * t.tiles);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.k_full[i], L::kConvWarps);
            mbar_init(&bar.v_full[i], L::kConvWarps);
            mbar_init(&bar.k_free[i], 1);
            mbar_init(&bar.v_free[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_done[i], 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&bar.sc_full[i], 1);
        mbar_init(&bar.raw_k_full, 1);
        mbar_init(&bar.raw_v_full, 1);
        mbar_init(&bar.raw_k_free, L::kConvWarps);
        mbar_init(&bar.raw_v_free, L::kConvWarps);
        mbar_init(&bar.fin, 1);
        fence_barrier_init();
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_slot, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // Not before the wait above (see KvAttnArgs::behind_tiles), and not before the Tensor Memory is
    // taken: a later kernel that took all of it and waited for this one would never see it end.
    grid_dep_launch();
    const uint32_t tbase = tmem_slot;

    if (warp < L::kSoftWarps) {
        softmax_role<BF16, DT>(a, t, qsm, sc, bar, tbase, abort);
    } else if (t.steps > 0) {
        if (warp < kMmaWarp)
            convert_role<F8, DT>(a, t, kraw, vraw, ksm, vsm, sc, bar, abort);
        else if (warp == kCopyWarp)
            copy_role<DT>(a, t, &km, &vm, kraw, vraw, sc, bar, abort);
        else if (lane == 0)
            mma_role<DT>(a, t, smem_u32(qsm), smem_u32(ksm), smem_u32(vsm), bar, tbase, abort);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tbase, kTmemCols);
}

struct TilesPlan {
    const void *fn;
    int rows, keys, smem;
};

template <bool F8, bool BF16, int DT>
TilesPlan tiles_plan()
{
    return {reinterpret_cast<const void *>(kv_attn_tiles_kernel<F8, BF16, DT>), Layout<DT>::kRows, Layout<DT>::kKeys,
            Layout<DT>::kBytes + 1024};
}

template <bool F8, bool BF16>
TilesPlan tiles_plan(int head_dim)
{
    return head_dim <= 64 ? tiles_plan<F8, BF16, 64>() : head_dim <= 128 ? tiles_plan<F8, BF16, 128>() : tiles_plan<F8, BF16, 256>();
}

}  // namespace

wq_status kv_attn_tiles(KvAttnArgs a, bool bf16, bool f8, cudaStream_t st)
{
    const TilesPlan p = f8 ? (bf16 ? tiles_plan<true, true>(a.head_dim) : tiles_plan<true, false>(a.head_dim))
                           : (bf16 ? tiles_plan<false, true>(a.head_dim) : tiles_plan<false, false>(a.head_dim));
    if (cudaFuncSetAttribute(p.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem) != cudaSuccess)
        return check_launch("cudaFuncSetAttribute(kv_attn_tiles_kernel)");
    // whichever makes fewer blocks
    const int64_t by_seq = kv_row_item(a.M, a.n_seqs, a.group, p.rows), by_rows = kv_row_item(a.M, 0, a.group, p.rows, a.few_rows);
    a.by_rows = by_rows < by_seq ? a.few_rows : 0;
    const int64_t blocks = std::min(by_seq, by_rows) * a.kv_heads;
    if (blocks > 0x7fffffff) return fail(WQ_ERR_INVALID_ARG, "too many blocks: fewer rows or heads a call");
    CUtensorMap km, vm;
    wq_status rc = encode_cache(&km, &vm, a, std::min(1 << a.page_shift, p.keys));
    if (rc != WQ_OK) return rc;
    PreparedLaunch L;
    set_attn_launch(L, p.fn, unsigned(blocks), kThreads, size_t(p.smem), km, vm, a);
    return launch_prepared(L, st, "kv_attn_tiles_kernel");
}

}  // namespace wq
