// wq_kv_tiles.cu -- kv_attention for many rows per key head (prefill): 256 rows a block on the
// 5th-generation tensor cores (tcgen05).
//
// Mathematics (as in wq_kv_attn.cu): S = Q Kc^T per block of 128 keys, x = S * (ks * sm_scale *
// log2 e), running maximum m and weight sum l in binary32, P = 2^(x - m) * vs / vref in binary16,
// O += P Vc, out = O * vref / l.  Codes are exact in binary16.  vref is a power of two above
// every value scale so far, so that P fits binary16 whatever the scales are.
//
// Bound by the tensor cores and by the 32 x 1024 exponentials of a 256 x 128 block, which cost
// about as much; so the two 128-row tiles of a block take turns: while one tile's products run,
// the other tile's softmax does.
//  * warps 0-3 / 4-7: tile 0 / 1, a thread per row: query row to shared memory, then per key
//    block: scores from Tensor Memory (twice: maximum, then weights), weights back over them as
//    the A operand of the second product.  O stays in Tensor Memory; it is rescaled only when the
//    maximum rose by more than 2^kSlack or a larger value scale arrived, which is rare after the
//    first blocks.
//  * warps 8-15: codes of the next block from global memory (in flight in registers while the
//    block before is worked on), widened to binary16 into the 128-byte swizzled layout of the
//    MMA's K-major operands: keys as rows of dimensions, values transposed as rows of keys.
//  * warp 16: one thread issues the MMAs.
// Every wait is bounded; on expiry the block records an error, stops and frees its Tensor Memory.
#include <cuda_runtime.h>
#include <stdint.h>

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
constexpr int kRows = 2 * kTile;     // rows of a block
constexpr int kKeys = 128;           // keys of a step
constexpr int kGroups = kKeys / 16;  // a group of 16 keys lies in one page
constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kThreads = 32 * (kSoftWarps + kConvWarps + 1);
constexpr int kRing = 4;             // scale sets: a set is rewritten once both tiles are two steps on
constexpr uint32_t kTmemCols = 512, kScol = 0, kOcol = 256;  // two 128-column tiles of each

// A maximum that rises by less than 2^kSlack is not followed, so weights reach 2^kSlack; raised
// by 2^kRaise they reach 2^15 in binary16, and are exact to half a step down to 2^-(14 + kRaise).
constexpr float kSlack = 4.f, kRaise = 11.f;

struct Bars {
    uint64_t q_full, k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_done[2], sc_full[kRing], fin;
};
struct Scales {
    float k[kRing][kGroups], v[kRing][kGroups];
    uint32_t dead[kRing];  // groups whose block-table entry is no page
};

template <int DT>
struct Layout {
    static constexpr int kAtom = 128 * 128;            // 128 rows of 64 binary16
    static constexpr int kQ = DT / 64 * kAtom;         // a query tile, a key step
    static constexpr int kV = 2 * DT * 128;            // DT rows of 128 keys
    static constexpr int kBytes = 2 * kQ + 2 * kQ + 2 * kV;
};

__device__ __forceinline__ uint64_t globaltimer()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits at most about 2 s, or until another role gave up.  wait_warp: the whole warp, with one
// answer, so that a warp gives up together.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait_short(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_short(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > 2000000000ull) {
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

__device__ __forceinline__ uint32_t ldg32(const uint8_t *p) { return __ldg(reinterpret_cast<const uint32_t *>(p)); }
__device__ __forceinline__ uint4 ldg128(const uint8_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

struct Item {
    KvSpan s;
    int b, head, row0, rows;  // the block's rows
    int keys;                 // keys that its last row sees
    int steps, tiles;
};

// ------------------------------------------------------------------ codes to binary16
template <bool F8, int DT>
__device__ void convert_role(const KvAttnArgs &a, const Item &t, uint8_t *ksm, uint8_t *vsm, Scales &sc, Bars &bar,
                             volatile int *abort)
{
    constexpr int kPerRow = DT / 16;                  // 16-byte chunks of a key
    constexpr int kPass = kConvThreads / kPerRow;     // keys of a pass
    constexpr int kKp = kKeys / kPass;                // passes: 4 (DT 128) or 2
    constexpr int kVt = DT / 64;                      // value tasks (8 keys x 4 dimensions) of a thread
    const int ct = threadIdx.x - 32 * kSoftWarps, cw = ct / 32, lane = ct % 32;
    const int32_t *table = a.block_table + int64_t(t.b) * a.max_pages;
    const int last_page = (t.keys - 1) >> a.page_shift, slot_mask = (1 << a.page_shift) - 1;
    const int chunk = ct % kPerRow, krow = ct / kPerRow;
    // values: a warp takes 32 keys x 32 dimensions; lanes so that both the 32-byte reads and the
    // transposed 16-byte stores are free of conflicts
    const int tg = lane % 8 / 2, dg = 2 * (lane / 8) + lane % 2;
    auto entry_of = [&](int key) { return __ldg(table + min(key >> a.page_shift, last_page)); };
    auto row_of = [&](int entry, int key) {
        const int64_t page = kv_page_ok(entry, a.num_pages);
        return kv_code_offset(page < 0 ? 0 : page, t.head, key & slot_mask, a.kv_heads, a.page_shift, a.pitch);
    };
    uint4 kraw[kKp];
    uint32_t vraw[kVt][8];
    int kent[kKp], vent[kVt], sent = 0;
    float ks = 0.f, vs = 0.f;
    bool sbad = false;
    auto v_key = [&](int i) { return 32 * ((cw + 8 * i) % 4) + 8 * tg; };
    auto v_dim = [&](int i) { return 32 * ((cw + 8 * i) / 4) + 4 * dg; };
    auto load_entries = [&](int key0) {
#pragma unroll
        for (int i = 0; i < kKp; ++i) kent[i] = entry_of(key0 + krow + kPass * i);
#pragma unroll
        for (int i = 0; i < kVt; ++i) vent[i] = entry_of(key0 + v_key(i));
        if (ct < kGroups) sent = entry_of(key0 + 16 * ct);
    };
    auto load_k = [&](int key0) {
#pragma unroll
        for (int i = 0; i < kKp; ++i)
            kraw[i] = 16 * chunk < a.pitch ? ldg128(a.k + row_of(kent[i], key0 + krow + kPass * i) + 16 * chunk)
                                           : make_uint4(0, 0, 0, 0);
        if (ct < kGroups) {
            const int64_t page = kv_page_ok(sent, a.num_pages);
            sbad = page < 0 && key0 + 16 * ct < t.keys;
            const int64_t si = kv_scale_index(page < 0 ? 0 : page, t.head, a.kv_heads);
            ks = __ldg(a.k_scale + si);
            vs = page < 0 ? 0.f : __ldg(a.v_scale + si);
        }
    };
    auto load_v = [&](int key0) {
#pragma unroll
        for (int i = 0; i < kVt; ++i) {
            const int key = key0 + v_key(i), d = v_dim(i);
            const uint8_t *p = a.v + row_of(vent[i], key) + d;
            const bool bad = kv_page_ok(vent[i], a.num_pages) < 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // slots behind the last key hold anything, e4m3 NaN codes among it
                const bool dead = F8 && (bad || key + e >= t.keys);
                vraw[i][e] = d < a.pitch && !dead ? ldg32(p + e * a.pitch) : 0u;
            }
        }
    };
    load_entries(0);
    load_k(0);
    load_v(0);
    if (t.steps > 1) load_entries(kKeys);
    for (int j = 0; j < t.steps; ++j) {
        const int buf = j & 1;
        const bool more = j + 1 < t.steps;
        uint8_t *kb = ksm + buf * Layout<DT>::kQ, *vb = vsm + buf * Layout<DT>::kV;
        // ---- keys
        if (j >= 2 && !wait_warp(&bar.k_free[buf], ((j >> 1) - 1) & 1, abort)) return;
#pragma unroll
        for (int i = 0; i < kKp; ++i) {
            const int r = krow + kPass * i;
            uint32_t w[4] = {kraw[i].x, kraw[i].y, kraw[i].z, kraw[i].w};
            if constexpr (F8) {
                if (a.head_dim < a.pitch)  // bytes behind the head hold anything
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (16 * chunk + 4 * x >= a.head_dim) w[x] = 0u;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] ^= 0x80808080u;
            }
            uint8_t *row = kb + chunk / 4 * Layout<DT>::kAtom + r * 128;
            const uint4 lo = make_uint4(widen<F8, 0>(w[0]), widen<F8, 1>(w[0]), widen<F8, 0>(w[1]), widen<F8, 1>(w[1]));
            const uint4 hi = make_uint4(widen<F8, 0>(w[2]), widen<F8, 1>(w[2]), widen<F8, 0>(w[3]), widen<F8, 1>(w[3]));
            const int c = 2 * (chunk % 4);
            // the lanes of the upper 64 dimensions store their halves in the other order: the two
            // atoms share banks
            const bool swap = chunk >= 4;
            sts128(row + (((c + swap) ^ (r & 7)) << 4), swap ? hi : lo);
            sts128(row + (((c + !swap) ^ (r & 7)) << 4), swap ? lo : hi);
        }
        if (cw == 0) {
            const uint32_t dead = __ballot_sync(0xffffffffu, sbad) & ((1u << kGroups) - 1);
            if (lane < kGroups) {
                sc.k[j % kRing][lane] = ks * a.sm_scale * kLog2e;
                sc.v[j % kRing][lane] = vs;
            }
            if (lane == 0) {
                sc.dead[j % kRing] = dead;
                if (dead) atomicCAS(&g_kv_tiles_error, kErrNone, kErrRange);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sc_full[j % kRing]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.k_full[buf]);
        if (more) load_k((j + 1) * kKeys);
        // ---- values
        if (j >= 2 && !wait_warp(&bar.v_free[buf], ((j >> 1) - 1) & 1, abort)) return;
#pragma unroll
        for (int i = 0; i < kVt; ++i) {
            const int key = v_key(i), d = v_dim(i);
            uint32_t o[4][4];  // [dimension][pair of keys]
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t x = prmt(vraw[i][2 * e], vraw[i][2 * e + 1], 0x5140);
                uint32_t y = prmt(vraw[i][2 * e], vraw[i][2 * e + 1], 0x7362);
                if constexpr (!F8) {
                    x ^= 0x80808080u;
                    y ^= 0x80808080u;
                }
                o[0][e] = widen<F8, 0>(x);
                o[1][e] = widen<F8, 1>(x);
                o[2][e] = widen<F8, 0>(y);
                o[3][e] = widen<F8, 1>(y);
            }
            if (d < a.pitch) {
                uint8_t *base = vb + key / 64 * (DT * 128);
                const int c = key % 64 / 8;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sts128(base + (d + x) * 128 + ((c ^ ((d + x) & 7)) << 4), make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]));
            }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_full[buf]);
        if (more) load_v((j + 1) * kKeys);
        if (j + 2 < t.steps) load_entries((j + 2) * kKeys);
    }
}

// ------------------------------------------------------------------ MMA issue (one thread)
template <int DT>
__device__ void mma_role(const KvAttnArgs &a, const Item &t, uint32_t qaddr, uint32_t kaddr, uint32_t vaddr, Bars &bar,
                         uint32_t tbase, volatile int *abort)
{
    const uint32_t iqk = tc::idesc_f16(false, kTile, kKeys), ipv = tc::idesc_f16(false, kTile, a.pitch);
    const uint64_t dq = tc::sdesc_sw128(qaddr), dk = tc::sdesc_sw128(kaddr), dv = tc::sdesc_sw128(vaddr);
    const int ksteps = a.pitch / 16;
    auto qk = [&](int tile, int buf) {
        const uint64_t q = dq + uint64_t(tile * Layout<DT>::kQ >> 4), k = dk + uint64_t(buf * Layout<DT>::kQ >> 4);
        for (int i = 0; i < ksteps; ++i) {
            const uint64_t off = uint64_t(((i >> 2) * Layout<DT>::kAtom + (i & 3) * 32) >> 4);
            tc::mma_f16_ss(tbase + kScol + 128 * tile, q + off, k + off, iqk, i > 0);
        }
        tc::commit(&bar.s_full[tile]);
    };
    auto pv = [&](int tile, int buf, bool first) {
        const uint64_t v = dv + uint64_t(buf * Layout<DT>::kV >> 4);
#pragma unroll
        for (int i = 0; i < kKeys / 16; ++i) {
            const uint64_t off = uint64_t(((i >> 2) * (DT * 128) + (i & 3) * 32) >> 4);
            tc::mma_f16_ts(tbase + kOcol + 128 * tile, tbase + kScol + 128 * tile + 8 * i, v + off, ipv, !first || i > 0);
        }
        tc::commit(&bar.o_done[tile]);
    };
    if (!wait(&bar.q_full, 0, abort) || !wait(&bar.k_full[0], 0, abort)) return;
    tc::fence_after_sync();
    for (int tile = 0; tile < t.tiles; ++tile) qk(tile, 0);
    tc::commit(&bar.k_free[0]);
    bool ok = true;
    for (int j = 0; j < t.steps && ok; ++j) {
        const int buf = j & 1, nbuf = buf ^ 1;
        const bool more = j + 1 < t.steps;
        for (int tile = 0; tile < t.tiles; ++tile) {
            ok = wait(&bar.p_full[tile], j & 1, abort) && (tile || wait(&bar.v_full[buf], (j >> 1) & 1, abort));
            if (!ok) break;
            tc::fence_after_sync();
            pv(tile, buf, j == 0);
            if (more) {
                if (!tile) {
                    ok = wait(&bar.k_full[nbuf], ((j + 1) >> 1) & 1, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                }
                qk(tile, nbuf);  // behind the tile's second product in the pipe: it may overwrite the weights
            }
        }
        if (!ok) break;
        tc::commit(&bar.v_free[buf]);
        if (more) tc::commit(&bar.k_free[nbuf]);
    }
    tc::commit(&bar.fin);  // all MMAs complete before the Tensor Memory is freed
    wait(&bar.fin, 0, abort);
}

// ------------------------------------------------------------------ softmax (a thread per row)
template <bool BF16, int DT>
__device__ void softmax_role(const KvAttnArgs &a, const Item &t, uint8_t *qsm, const Scales &sc, Bars &bar,
                             uint32_t tbase, volatile int *abort)
{
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, tile = warp / 4;
    if (tile >= t.tiles) return;
    const int r = 32 * (warp % 4) + lane, row = tile * kTile + r;
    const bool live = row < t.rows;
    const int i = live ? (t.row0 + row) / a.group : 0, h = live ? (t.row0 + row) % a.group : 0;
    const int64_t at = (int64_t(t.s.q0 + i) * a.q_heads + t.head * a.group + h) * a.head_dim;
    const int seen = live ? t.s.len - t.s.n + i + 1 : 0;
    const uint32_t tlane = tbase + (uint32_t(32 * (warp % 4)) << 16);
    const uint32_t scol = tlane + kScol + 128 * tile, ocol = tlane + kOcol + 128 * tile;

    // ---- the query row, binary16 (bfloat16 rows scaled by a power of two, see load_queries)
    float unscale = 1.f;
    {
        const uint16_t *q = static_cast<const uint16_t *>(a.q) + at;
        float up = 1.f;
        if constexpr (BF16) {
            float amax = 0.f;
            for (int d = 0; d < a.head_dim && live; d += 4) {
                const uint2 x = *reinterpret_cast<const uint2 *>(q + d);
                const float2 lo = act_f2<T>(x.x), hi = act_f2<T>(x.y);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(lo.x), fabsf(lo.y)), fmaxf(fabsf(hi.x), fabsf(hi.y))));
            }
            const int e = kv_clamp(int(__float_as_uint(amax) >> 23) - 127, -120, 120);
            up = __uint_as_float(uint32_t(127 - e) << 23);
            unscale = __uint_as_float(uint32_t(127 + e) << 23);
        }
        uint8_t *base = qsm + tile * Layout<DT>::kQ + r * 128;
        for (int c = 0; c < DT / 8; ++c) {
            uint2 x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = 8 * c + 4 * k;
                x[k] = live && d < a.head_dim ? *reinterpret_cast<const uint2 *>(q + d) : make_uint2(0, 0);
                if constexpr (BF16) {
                    const float2 lo = act_f2<T>(x[k].x), hi = act_f2<T>(x[k].y);
                    x[k] = make_uint2(act_t2<__half>(lo.x * up, lo.y * up), act_t2<__half>(hi.x * up, hi.y * up));
                }
            }
            sts128(base + c / 8 * Layout<DT>::kAtom + (((c % 8) ^ (r & 7)) << 4), make_uint4(x[0].x, x[0].y, x[1].x, x[1].y));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_full);
    }

    float m = -INFINITY, l = 0.f, vref = 0.f;
    for (int j = 0; j < t.steps; ++j) {
        const int set = j % kRing, key0 = j * kKeys;
        if (!wait_warp(&bar.sc_full[set], (j / kRing) & 1, abort) || !wait_warp(&bar.s_full[tile], j & 1, abort)) return;
        tc::fence_after_sync();
        const uint32_t dead = sc.dead[set];
        const int left = seen - key0;  // keys of this step that the row sees
        const bool masked = __any_sync(0xffffffffu, left < kKeys) || dead;
        float kc[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) kc[g] = sc.k[set][g] * unscale;
        // ---- maximum
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            tc::ld_32x32b_x32(scol + 32 * c, s);
            tc::wait_ld();
            if (masked) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (32 * c + x < left && !(dead >> (2 * c + x / 16) & 1))
                        mx = fmaxf(mx, __uint_as_float(s[x]) * kc[2 * c + x / 16]);
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) mx = fmaxf(mx, __uint_as_float(s[x]) * kc[2 * c + x / 16]);
            }
        }
        const float m_new = mx > m + kSlack ? mx : m;  // -inf until the row sees a key
        // ---- reference of the value scales: a power of two above all so far
        float vmax = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) vmax = fmaxf(vmax, fabsf(sc.v[set][g]));
        const float vnew = vmax >= vref && vmax > 0.f
                               ? __uint_as_float((__float_as_uint(vmax) & 0x7f800000u) + 0x00800000u) : vref;
        const float inv = vnew > 0.f ? 1.f / vnew : 0.f;
        const float fm = m_new == m ? 1.f : exp2_approx(m - m_new);
        const float fo = vnew == vref ? fm : fm * (vref * inv);
        l *= fm;
        if (j > 0 && __any_sync(0xffffffffu, fo != 1.f)) {
            if (!wait_warp(&bar.o_done[tile], (j - 1) & 1, abort)) return;
            tc::fence_after_sync();
#pragma unroll
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
        m = m_new;
        vref = vnew;
        // ---- weights, over the scores that are already read
        const float base = m == -INFINITY ? 0.f : m - kRaise;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t s[32], p[16];
            tc::ld_32x32b_x32(scol + 32 * c, s);
            tc::wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
                const int g = 2 * c + x / 16;
                float w0 = exp2_approx(fmaf(__uint_as_float(s[x]), kc[g], -base));
                float w1 = exp2_approx(fmaf(__uint_as_float(s[x + 1]), kc[g], -base));
                if (masked) {
                    const bool gd = dead >> g & 1;
                    if (32 * c + x >= left || gd) w0 = 0.f;
                    if (32 * c + x + 1 >= left || gd) w1 = 0.f;
                }
                l += w0 + w1;
                const float v = sc.v[set][g] * inv;
                p[x / 2] = act_t2<__half>(w0 * v, w1 * v);
            }
            tc::st_32x32b_x16(scol + 16 * c, p);
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[tile]);
    }
    if (t.steps > 0 && !wait_warp(&bar.o_done[tile], (t.steps - 1) & 1, abort)) return;
    tc::fence_after_sync();
    const float inv = l > 0.f ? vref / l : (l == l ? 0.f : l);
    uint16_t *out = static_cast<uint16_t *>(a.out) + at;
#pragma unroll
    for (int c = 0; c < DT / 32; ++c) {
        uint32_t o[32];
        if (t.steps > 0) {
            tc::ld_32x32b_x32(ocol + 32 * c, o);
            tc::wait_ld();
        }
#pragma unroll
        for (int x = 0; x < 32; x += 4)
            if (live && 32 * c + x < a.head_dim) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = l == 0.f ? 0.f : __uint_as_float(o[x + e]) * inv;
                *reinterpret_cast<uint2 *>(out + 32 * c + x) = make_uint2(act_t2<T>(y[0], y[1]), act_t2<T>(y[2], y[3]));
            }
    }
}

template <bool F8, bool BF16, int DT>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_tiles_kernel(const __grid_constant__ KvAttnArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Bars bar;
    __shared__ Scales sc;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, s_seq[4];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qsm = smem, *ksm = qsm + 2 * Layout<DT>::kQ, *vsm = ksm + 2 * Layout<DT>::kQ;
    volatile int *abort = &abort_flag;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    grid_dep_launch();
    grid_dep_wait();  // queries, cache and batch arrays may come from the kernel before

    const int64_t item = blockIdx.x / a.kv_heads;
    if (tid == 0) {
        s_seq[0] = -1;
        abort_flag = 0;
    }
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int lo = a.cu_q[b], hi = a.cu_q[b + 1], len = a.seq_len[b];
        const KvSpan s = kv_span(lo, hi, len, a.M, a.capacity);
        if (kv_row_item(s.q0, b, a.group, kRows) <= item && item < kv_row_item(s.q0 + s.n, b + 1, a.group, kRows)) {
            s_seq[0] = b;
            s_seq[1] = lo;
            s_seq[2] = hi;
            s_seq[3] = len;
        }
    }
    __syncthreads();
    Item t;
    t.b = s_seq[0];
    if (t.b < 0) return;
    t.s = kv_span(s_seq[1], s_seq[2], s_seq[3], a.M, a.capacity);
    if (tid == 0 && s_seq[3] > a.capacity) atomicCAS(&g_kv_tiles_error, kErrNone, kErrRange);
    const int all = t.s.n * a.group;
    // the last rows first: they see the most keys
    const int64_t k = kv_tiles(t.s.n, a.group, kRows) - 1 - (item - kv_row_item(t.s.q0, t.b, a.group, kRows));
    if (k < 0 || all <= a.few_rows) return;
    t.head = blockIdx.x % a.kv_heads;
    t.row0 = int(k) * kRows;
    t.rows = min(kRows, all - t.row0);
    t.keys = max(0, t.s.len - t.s.n + (t.row0 + t.rows - 1) / a.group + 1);
    t.steps = (t.keys + kKeys - 1) / kKeys;
    t.tiles = t.rows > kTile ? 2 : 1;

    if (tid == 0) {
        mbar_init(&bar.q_full, 4 * t.tiles);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.k_full[i], kConvWarps);
            mbar_init(&bar.v_full[i], kConvWarps);
            mbar_init(&bar.k_free[i], 1);
            mbar_init(&bar.v_free[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_done[i], 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&bar.sc_full[i], 1);
        mbar_init(&bar.fin, 1);
        fence_barrier_init();
    }
    if (warp == kSoftWarps + kConvWarps) {
        tc::tmem_alloc(&tmem_slot, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = tmem_slot;

    if (warp < kSoftWarps) {
        softmax_role<BF16, DT>(a, t, qsm, sc, bar, tbase, abort);
    } else if (t.steps > 0) {
        if (warp < kSoftWarps + kConvWarps)
            convert_role<F8, DT>(a, t, ksm, vsm, sc, bar, abort);
        else if (lane == 0)
            mma_role<DT>(a, t, smem_u32(qsm), smem_u32(ksm), smem_u32(vsm), bar, tbase, abort);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kSoftWarps + kConvWarps) tc::tmem_dealloc(tbase, kTmemCols);
}

template <bool F8, bool BF16>
const void *tiles_kernel(bool small)
{
    return small ? reinterpret_cast<const void *>(kv_attn_tiles_kernel<F8, BF16, 64>)
                 : reinterpret_cast<const void *>(kv_attn_tiles_kernel<F8, BF16, 128>);
}

}  // namespace

wq_status kv_attn_tiles(const KvAttnArgs &a, bool bf16, bool f8, cudaStream_t st)
{
    const bool small = a.head_dim <= 64;
    const void *fn = f8 ? (bf16 ? tiles_kernel<true, true>(small) : tiles_kernel<true, false>(small))
                        : (bf16 ? tiles_kernel<false, true>(small) : tiles_kernel<false, false>(small));
    // the most that any sequence of the call leaves for its Tensor Memory: one block an SM
    const int smem = 1024 + (small ? Layout<64>::kBytes : Layout<128>::kBytes);
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return check_launch("cudaFuncSetAttribute(kv_attn_tiles_kernel)");
    const int64_t blocks = kv_row_item(a.M, a.n_seqs, a.group, kRows) * a.kv_heads;
    if (blocks > 0x7fffffff) return fail(WQ_ERR_INVALID_ARG, "too many blocks: fewer rows or heads a call");
    PreparedLaunch L;
    L.set(fn, dim3(unsigned(blocks)), dim3(kThreads), size_t(smem), a);
    return launch_prepared(L, st, "kv_attn_tiles_kernel");
}

}  // namespace wq
