// Attention of many streams' queries over pages that the streams share, on the
// fifth-generation tensor cores: the shared rows are read once for all of them.
//
// Rows: the query columns of a group's streams on one KV head, token after
// token, 256 to an M-tile.  No row is masked (every query of the group comes
// behind the shared positions).  A pair of CTAs (cta_group::2) takes an M-tile
// and a range of keys, in tiles of 128: each CTA holds half of the rows, half of
// a tile's K (64 keys) and half of its V (128 dims), so a tile's bytes go into
// shared memory once for 256 rows.  Per tile:
//   S = Q K^T -> TMEM (Q sits there too), P = softmax numerators in fp16 ->
//   shared memory, O += P V -> TMEM
// with V as fp16: bf16 rows are converted where they lie, e4m3 codes (K's too)
// on their way from a raw ring, both exactly (bf16 from 2^-14 on).  So the PV
// product takes one P part of 11 significant bits.  The scales of e4m3 rows go
// into the scores (K) and the weights (V); the weights' reference is the running
// maximum of score + V-scale exponent, so that they stay in fp16's range
// wherever the scales lie.
//   warps 0-7   softmax: two threads a row, each on 64 of a tile's keys
//   warps 8, 9  copy K and V (halves of one page, of 16-row runs, or key by key)
//   warps 10-13 convert
//   warp 14     first CTA: issues S; second: passes on that its K is there
//   warp 15     first CTA: issues PV
// The splits' O, maxima and sums go to the workspace; prefix_combine merges them
// with the partials of the streams' own positions (pkv_window.cu).
#include <algorithm>
#include <cfloat>

#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kN = 128;        // keys a tile
constexpr int kRows = 2 * kM;  // rows of an M-tile
constexpr int kThreads = 512;
constexpr int kSoftWarps = 8, kWarpK = 8, kWarpV = 9, kWarpConv = 10, kConvWarps = 4, kWarpS = 14, kWarpPv = 15;
constexpr uint32_t kTmemCols = 512, kQCol = 0, kSCol = 128, kOCol = 256;
constexpr int kSlotBytes = 32768;  // 64 K rows, or 128 half V rows, of 16-bit elements
constexpr int kRawBytes = 16384;   // the same of codes
constexpr int kKRegion = 64 * 128;   // one 64-dim region of 64 K rows
constexpr int kVRegion = 128 * 128;  // one 64-dim region of 128 V rows
constexpr int kPRegion = kM * 128;   // 64 keys of the CTA's 128 P rows
constexpr float kScaleLog2 = 0.0625f * 1.4426950408889634f;  // log2(e) / sqrt(256)
constexpr float kRescale = 8.f;          // rescale O when the reference grows by more than 2^8
constexpr float kFarScore = 67108864.f;  // 2^26: references beyond it are reported (float32 steps of 4 there)

template <bool kFp8>
struct Lay {
    static constexpr int slots = kFp8 ? 2 : 3;      // of 16-bit K, and of V
    static constexpr int raw = kFp8 ? 3 : 0;        // of codes, K and V in turn
    static constexpr int off_k = 2 * kPRegion;      // P before it
    static constexpr int off_v = off_k + slots * kSlotBytes;
    static constexpr int off_raw = off_v + slots * kSlotBytes;
    static constexpr int off_red = off_raw + raw * kRawBytes;  // [parity][half][row]
    static constexpr int off_scl = off_red + 2 * 2 * kM * 4;   // [tile parity][K scale, V exponent, V scale][key]
    static constexpr int off_bar = off_scl + (kFp8 ? 2 * 3 * kN * 4 : 0);
    // barriers.  Of the first CTA, with arrivals from both: k_ready, v_ready,
    // q_full, s_empty, p_full.  Of each CTA: the others.
    static constexpr int k_full = 0, v_full = 3;      // copies landed (codes: the raw ring's, in k_full)
    static constexpr int raw_free = 6;                // a raw slot is converted
    static constexpr int k_ready = 9, v_ready = 12;   // a slot may be multiplied
    static constexpr int k_free = 15, v_free = 18;    // its products are done
    static constexpr int q_full = 21, s_full = 22, s_empty = 23, p_full = 24, o_done = 25;
    static constexpr int red = 26;                    // a row quarter's exchange (4)
    static constexpr int scl_full = 30, scl_free = 32;
    static constexpr int drain = 34;
    static constexpr int bars = 36;
    static constexpr int smem = off_bar + bars * 8 + 16;
    static_assert(smem <= 232448, "above the 227 KB a CTA may hold");
};

struct PrefixArgs {
    const uint16_t *q;
    float *ws;
    uint32_t *status;
    int32_t n_groups, n_kv_heads, n_q_heads, group;  // group: query heads of a KV head
    PrefixGroup g[kMaxGroups];
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void arrive_first(uint64_t *bar) {  // at the first CTA's barrier
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(bar, 0)) : "memory");
}
// mbar_wait for what the other CTA arrived at, too.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, uint32_t *status) {
    const auto test = [&]() -> bool {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (test()) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t spin = 0;; ++spin) {
        if (test()) return true;
        if ((spin & 255u) == 255u && global_ns() - t0 > kWaitLimitNs) {
            if (status) atomicOr(status, PKV_DEV_TIMEOUT);
            return false;
        }
    }
}

// A pair's work.
struct Work {
    int g, kvh, split;
    int first, count;  // the CTA's rows of the group
    int key0, key1, ntiles;
};
__device__ __forceinline__ Work work_of(const PrefixArgs &a, int item, int rank) {
    Work w;
    w.g = find_seq(a.n_groups, item, [&](int t) { return a.g[t].work_off; });
    const PrefixGroup &g = a.g[w.g];
    const int mtiles = (g.rows + kRows - 1) / kRows, r = item - g.work_off, u = r / mtiles;
    const int row0 = (r - u * mtiles) * kRows, rows = min(kRows, g.rows - row0), half = (rows + 1) >> 1;
    w.kvh = u / g.nsplit;
    w.split = u - w.kvh * g.nsplit;
    w.first = row0 + rank * half;
    w.count = rank ? rows - half : half;
    w.key0 = w.split * g.split_tiles * kN;
    w.key1 = min(g.len, w.key0 + g.split_tiles * kN);
    w.ntiles = (w.key1 - w.key0 + kN - 1) / kN;
    return w;
}

// Where a tile's rows are.  With a map: lane i & 7 has run i of 16 rows; without,
// lane i keys i, i + 32, i + 64, i + 96.  Keys behind the end are the last run's
// or the last key's (their scores are masked, their rows finite).
struct Look {
    int64_t at[4];  // element offset of the page from layer_base
    int row[4];     // row in it
};

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_partial(const __grid_constant__ DecodeMaps maps, const __grid_constant__ PrefixArgs a) {
    using L = Lay<kFp8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::off_bar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::bars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cta_rank());
    {
        // the address as the hardware gives it; the same in both CTAs
        uint32_t base;
        asm volatile("mov.u32 %0, %1;" : "=r"(base) : "r"(smem_u32(smem)));
        if (base & 1023u) {  // every thread of the pair returns before any barrier
            if (tid == 0 && a.status) atomicOr(a.status, PKV_DEV_SMEM);
            return;
        }
    }
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bars[L::k_full + i], 1);
            mbar_init(&bars[L::v_full + i], 1);
            mbar_init(&bars[L::raw_free + i], kConvWarps);
            mbar_init(&bars[L::k_ready + i], kFp8 ? 2 * kConvWarps : 1);
            mbar_init(&bars[L::v_ready + i], 2 * kConvWarps);
            mbar_init(&bars[L::k_free + i], 1);
            mbar_init(&bars[L::v_free + i], 1);
        }
        mbar_init(&bars[L::q_full], 2 * kSoftWarps);
        mbar_init(&bars[L::s_full], 1);
        mbar_init(&bars[L::s_empty], 2 * kSoftWarps);
        mbar_init(&bars[L::p_full], 2 * kSoftWarps);
        mbar_init(&bars[L::o_done], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bars[L::red + i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[L::scl_full + i], 2);
            mbar_init(&bars[L::scl_free + i], kSoftWarps);
            mbar_init(&bars[L::drain + i], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
        // prefix_combine may start: it waits for this grid
        pdl_trigger();
    }
    if (warp == kWarpS) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, sbase = smem_u32(smem);
    const Work w = work_of(a, static_cast<int>(blockIdx.x >> 1), rank);
    const PrefixGroup &g = a.g[w.g];
    const int H = a.n_kv_heads, G = a.group;

    auto wait = [&](int bar, uint32_t phase) -> bool {
        const bool ok = mbar_wait(&bars[bar], phase & 1, a.status);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    auto wait_warp = [&](int bar, uint32_t phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };
    auto wait_both = [&](int bar, uint32_t phase) -> bool {
        const bool ok = wait_cluster(&bars[bar], phase & 1, a.status);
        if (!ok) *abort_flag = 1;
        return ok;
    };

    // No grid-dependency wait before anything is read: the kernel before this one
    // on the stream (the streams' own positions, window_partial) lets this grid
    // start only behind its own wait, when everything queued before it is
    // visible, and itself writes no shared row, no query and none of these
    // partials.  Its end is waited for at this kernel's (the combine reads it).
    if (warp < kSoftWarps) {
        // ---------------- softmax ----------------
        const int r = lane + 32 * (warp & 3), hf = warp >> 2;
        const bool row_ok = r < w.count, active = 32 * (warp & 3) < w.count;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float *const red = reinterpret_cast<float *>(smem + L::off_red);
        uint32_t rc = 0;  // exchanges with the row's other thread so far
        bool ok = true;
        // the row's other thread's value of what it put beside this one
        auto exchange = [&](float v, float &other) -> bool {
            red[((rc & 1) * 2 + hf) * kM + r] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::red + (warp & 3)]);
            if (!wait_warp(L::red + (warp & 3), rc)) return false;
            other = red[((rc & 1) * 2 + (hf ^ 1)) * kM + r];
            ++rc;
            return true;
        };
        float qs = kScaleLog2;  // what a raw score is scaled by
        if (active) {
            const int gr = w.first + r, tok = row_ok ? gr / G : 0, h = row_ok ? gr - tok * G : 0;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.q + (((int64_t)g.tok0 + tok) * a.n_q_heads + w.kvh * G + h) * kHeadDim + 128 * hf);
            float dn = 1.f;
            if constexpr (kFp8) {
                // bf16 has the wider range: a power of two takes the row's largest
                // element to 2^14 .. 2^15, exactly, and goes into the scores' scale
                uint32_t top = 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint4 v = row_ok ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                 __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                }
                const uint32_t mine = max(top >> 16, top & 0xffffu);
                float other = 0.f;
                ok = exchange(__uint_as_float(mine), other);
                const int ex = static_cast<int>(max(mine, __float_as_uint(other)) >> 7);  // biased exponent
                // (zeros, and rows with an infinity or NaN, stay as they are)
                const int e = ex == 0 || ex == 0xff ? 0 : max(ex - 127 - 14, -100);
                dn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                qs = kScaleLog2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            }
#pragma unroll 1
            for (int h32 = 0; h32 < 2; ++h32) {
                uint32_t qv[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = row_ok ? __ldg(src + 8 * h32 + i) : make_uint4(0, 0, 0, 0);
                    const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        qv[4 * i + k] = kFp8 ? pack_f16(dn * bf16_lo(e[k]), dn * bf16_hi(e[k])) : e[k];
                }
                __syncwarp();
                tmem_st32(lane_base + kQCol + 64 * hf + 32 * h32, qv);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bars[L::q_full]);
        float m_used = -INFINITY, l = 0.f;
        uint8_t *const p_row = smem + hf * kPRegion + r * 128;
        for (int n = 0; ok && n < w.ntiles; ++n) {
            if (!(ok = wait_warp(L::s_full, n))) break;
            if (!active) {  // no row of the warp: S and P are nobody's
                if (lane == 0) arrive_first(&bars[L::s_empty]);
                if (n > 0 && !(ok = wait_warp(L::o_done, n - 1))) break;
                if (lane == 0) {
                    arrive_first(&bars[L::p_full]);
                    if (kFp8) mbar_arrive(&bars[L::scl_free + (n & 1)]);
                }
                __syncwarp();
                continue;
            }
            tc_fence_after();
            float x[64];
            {
                uint32_t sv[64];
                tmem_ld64(lane_base + kSCol + 64 * hf, sv);
#pragma unroll
                for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(sv[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first(&bars[L::s_empty]);
            const float *const scl = reinterpret_cast<const float *>(smem + L::off_scl) + (n & 1) * 3 * kN + 64 * hf;
            if constexpr (kFp8) {
                if (!(ok = wait_warp(L::scl_full + (n & 1), n >> 1))) break;
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 k = *reinterpret_cast<const float4 *>(scl + j);
                    x[j] *= k.x * qs;
                    x[j + 1] *= k.y * qs;
                    x[j + 2] *= k.z * qs;
                    x[j + 3] *= k.w * qs;
                }
            }
            const int kt = w.key0 + n * kN + 64 * hf;
            if (kt + 64 > w.key1) {  // the prefix's end: uniform
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (kt + j >= w.key1) x[j] = -INFINITY;
            }
            // this half's reference as eight interleaved chains, then the row's
            float m8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) m8[j] = -INFINITY;
            if constexpr (kFp8) {
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 e = *reinterpret_cast<const float4 *>(scl + kN + j);
                    m8[j & 7] = fmaxf(m8[j & 7], x[j] + e.x);
                    m8[(j + 1) & 7] = fmaxf(m8[(j + 1) & 7], x[j + 1] + e.y);
                    m8[(j + 2) & 7] = fmaxf(m8[(j + 2) & 7], x[j + 2] + e.z);
                    m8[(j + 3) & 7] = fmaxf(m8[(j + 3) & 7], x[j + 3] + e.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) m8[j & 7] = fmaxf(m8[j & 7], x[j]);
            }
            const float lmx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
            float omx = 0.f;
            if (!(ok = exchange(lmx, omx))) break;
            const float mx = fmaxf(lmx, omx) * (kFp8 ? 1.f : kScaleLog2);  // log2 units
            const bool grow = m_used != -INFINITY && mx > m_used + kRescale;
            if (__any_sync(0xffffffffu, grow)) {
                // correct this thread's half of O: the last tile's product first
                if (!(ok = wait_warp(L::o_done, n - 1))) break;
                tc_fence_after();
                const float m_new = fmaxf(m_used, mx);
                const float alpha = m_used == -INFINITY ? 0.f : ex2(m_used - m_new);
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + kOCol + 128 * hf + ch * 32, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                    tmem_st32(lane_base + kOCol + 128 * hf + ch * 32, o);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                l *= alpha;
                m_used = m_new;
            } else if (m_used == -INFINITY) {
                m_used = mx;  // nothing accumulated yet
            }
            // p = 2^(score - m): fp16 weights of 11 significant bits, at most 2^8
            // with the lazy rescale (times a V scale's mantissa below 2)
            const float m_off = m_used == -INFINITY ? 0.f : m_used;
            uint32_t p16[32];
            if constexpr (kFp8) {
                float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(scl + 2 * kN + j);
                    const float p0 = ex2(x[j] - m_off), p1 = ex2(x[j + 1] - m_off);
                    const float p2 = ex2(x[j + 2] - m_off), p3 = ex2(x[j + 3] - m_off);
                    ps[0] += p0;
                    ps[1] += p1;
                    ps[2] += p2;
                    ps[3] += p3;
                    p16[j / 2] = pack_f16(p0 * v.x, p1 * v.y);
                    p16[j / 2 + 1] = pack_f16(p2 * v.z, p3 * v.w);
                }
                l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::scl_free + (n & 1)]);
            } else {
                const float2 scale = make_float2(kScaleLog2, kScaleLog2), off = make_float2(-m_off, -m_off);
                float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float2 p = fma2(make_float2(x[j], x[j + 1]), scale, off);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    ps[(j >> 1) & 1] = add2(ps[(j >> 1) & 1], p);
                    p16[j / 2] = pack_f16(p.x, p.y);
                }
                l += (ps[0].x + ps[1].x) + (ps[0].y + ps[1].y);
            }
            // the P rows are free once the last tile's product is done
            if (n > 0 && !(ok = wait_warp(L::o_done, n - 1))) break;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4 *>(p_row + ((ch ^ (r & 7)) << 4)) =
                    make_uint4(p16[4 * ch], p16[4 * ch + 1], p16[4 * ch + 2], p16[4 * ch + 3]);
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first(&bars[L::p_full]);
        }
        // ---------------- the split's sums to the workspace ----------------
        if (ok && active) {
            float other = 0.f;
            ok = wait_warp(L::o_done, w.ntiles - 1) && exchange(l, other);
            l += other;
            tc_fence_after();
        }
        if (ok && active) {
            float *const acc = a.ws + g.ws_off;
            float *const ml = acc + (int64_t)H * g.nsplit * g.rows * kHeadDim;
            const int64_t prow = ((int64_t)w.kvh * g.nsplit + w.split) * g.rows + w.first + r;
            const int64_t mine = row_ok ? prow : -1;
            int64_t row[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) row[j] = shfl64(mine, (lane & ~3) + j);
            float2 odd = make_float2(0.f, 0.f);  // NaN once a sum is not finite
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(lane_base + kOCol + 128 * hf + 32 * ch, o);
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    odd = fma2(make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), make_float2(0.f, 0.f), odd);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = make_uint4(o[16 * h + 4 * j], o[16 * h + 4 * j + 1], o[16 * h + 4 * j + 2], o[16 * h + 4 * j + 3]);
                    quad_transpose(v, lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (row[j] >= 0)
                            *(reinterpret_cast<uint4 *>(acc + row[j] * kHeadDim + 128 * hf + 32 * ch + 16 * h) + (lane & 3)) = v[j];
                }
            }
            if (row_ok) {
                if (hf == 0) *reinterpret_cast<float2 *>(ml + 2 * prow) = make_float2(m_used, l);
                if ((odd.x + odd.y != 0.f || (m_used != -INFINITY && fabsf(m_used) > kFarScore)) && a.status)
                    atomicOr(a.status, PKV_DEV_RANGE);
            }
        }
    } else if (warp == kWarpK || warp == kWarpV) {
        // ---------------- copies ----------------
        const bool is_v = warp == kWarpV;
        const int ptok = g.ptok, n_pages = g.n_pages, n_table = (g.len + ptok - 1) / ptok;
        const int32_t *const table = g.table;
        const uint64_t pol = policy_evict_normal();  // the other M-tiles read the same rows
        const void *const map = g.map_run >= 0 ? &maps.map[g.map_run] : nullptr;
        const int whole_map = is_v ? g.map_v : g.map_k;
        const void *const map_w = whole_map >= 0 ? &maps.map[whole_map] : nullptr;
        const uint8_t *const base = reinterpret_cast<const uint8_t *>(g.layer_base);
        const bool runs = map != nullptr;
        auto look = [&](int m) -> Look {
            Look k;
            const int kt = w.key0 + m * kN;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                k.at[i] = 0;
                k.row[i] = 0;
                if (runs && i > 0) continue;
                const int last = runs ? w.key1 - 16 : w.key1 - 1;
                const int key = min(kt + (runs ? 16 * (lane & 7) : 32 * i + lane), last);
                const int page = key / ptok;
                k.row[i] = key - page * ptok;
                const int id = page < n_table ? __ldg(table + page) : -1;
                if (static_cast<uint32_t>(id) < static_cast<uint32_t>(n_pages)) {
                    k.at[i] = (int64_t)id * g.ps;
                } else if (!is_v && a.status) {
                    atomicOr(a.status, PKV_DEV_BAD_PAGE);
                }
            }
            return k;
        };
        // byte offset of a 16-bit or code row from layer_base
        auto row_bytes = [&](int64_t at, int row) -> int64_t {
            return kFp8 ? 2 * at + off8_code(is_v, H, ptok, w.kvh, row)
                        : 2 * (at + (is_v ? off_v(H, ptok, w.kvh, row) : off_k(ptok, w.kvh, row)));
        };
        // e4m3: the scales of keys lane, lane + 32, ... of a looked-up tile
        auto scales = [&](const Look &k, float (&s)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t at;
                int row;
                if (runs) {
                    const int src = 2 * i + (lane >> 4);
                    at = shfl64(k.at[0], src);
                    row = __shfl_sync(0xffffffffu, k.row[0], src) + (lane & 15);
                } else {
                    at = k.at[i];
                    row = k.row[i];
                }
                s[i] = __ldg(reinterpret_cast<const float *>(base + 2 * at + off8_scale(is_v, H, ptok, w.kvh, row)));
            }
        };
        float s_now[4] = {0.f, 0.f, 0.f, 0.f};
        Look now = look(0);
        if constexpr (kFp8) scales(now, s_now);
        int last_q = -1;
        bool ok = true;
        for (int m = 0; ok && m < w.ntiles; ++m) {
            Look next = now;
            if (m + 1 < w.ntiles) next = look(m + 1);
            // the slot
            const uint32_t q = kFp8 ? 2 * m + is_v : m;
            const uint32_t n_slots = kFp8 ? L::raw : L::slots, slot = q % n_slots;
            if (q >= n_slots &&
                !(ok = wait_warp((kFp8 ? L::raw_free : is_v ? L::v_free : L::k_free) + slot, q / n_slots - 1)))
                break;
            uint64_t *const full = &bars[(kFp8 || !is_v ? L::k_full : L::v_full) + slot];
            uint8_t *const dst = smem + (kFp8 ? L::off_raw + slot * kRawBytes : (is_v ? L::off_v : L::off_k) + slot * kSlotBytes);
            if (runs) {
                const int64_t rb = row_bytes(now.at[0], now.row[0]);
                const int y = static_cast<int>(g.layer_row + rb / (kFp8 ? 256 : 512));
                if (lane == 0) mbar_arrive_expect_tx(full, kFp8 ? kRawBytes : kSlotBytes);
                const int y0 = __shfl_sync(0xffffffffu, y, 0);  // (and the expected bytes come first)
                if (map_w) {
                    // the tile lies in one page: one copy (two of K's code halves)
                    if (kFp8) {
                        if (lane < (is_v ? 1 : 2))
                            tma_load_2d(dst + lane * 8192, map_w, is_v ? 128 * rank : 128 * lane, is_v ? y0 : y0 + 64 * rank, full, pol);
                    } else if (lane == 0) {
                        tma_load_3d(dst, map_w, 0, is_v ? y0 : y0 + 64 * rank, is_v ? 2 * rank : 0, full, pol);
                    }
                } else {
                    // 16-row runs, one box a lane: K four runs of all dims, V eight of half
                    const int nc = kFp8 ? (is_v ? 1 : 2) : (is_v ? 2 : 4);  // boxes of a run
                    const int rn = lane / nc, ch = lane - rn * nc, n_runs = is_v ? 8 : 4;
                    const int yr = __shfl_sync(0xffffffffu, y, (is_v ? rn : 4 * rank + rn) & 7);
                    if (rn < n_runs) {
                        if (kFp8)
                            tma_load_2d(dst + ch * 8192 + rn * 2048, map, is_v ? 128 * rank : 128 * ch, yr, full, pol);
                        else
                            tma_load_2d(dst + ch * (is_v ? kVRegion : kKRegion) + rn * 2048, map, 64 * (is_v ? 2 * rank + ch : ch),
                                        yr, full, pol);
                    }
                }
                __syncwarp();
            } else {
                // key by key: 16-byte chunks through the same swizzle
                int64_t src[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) src[i] = row_bytes(now.at[i], now.row[i]);
                constexpr int kChunks = kFp8 ? 16 : 32;  // of a row
                const int per = is_v ? kChunks / 2 : kChunks, rows_pass = 32 / per, n_rows = is_v ? 128 : 64;
                const int c = lane % per, sub = lane / per;
                const int region = is_v ? 128 * 128 : 64 * 128;
#pragma unroll 4
                for (int r0 = 0; r0 < n_rows; r0 += rows_pass) {
                    const int r = r0 + sub, key = (is_v ? 0 : 64 * rank) + r, i = key >> 5;
                    // (the four values by selects: an index would put them in memory)
                    const int64_t s0 = shfl64(src[0], key & 31), s1 = shfl64(src[1], key & 31);
                    const int64_t s2 = shfl64(src[2], key & 31), s3 = shfl64(src[3], key & 31);
                    const int64_t s = i == 0 ? s0 : i == 1 ? s1 : i == 2 ? s2 : s3;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     smem_u32(dst + (c >> 3) * region + r * 128 + (((c & 7) ^ (r & 7)) << 4))),
                                 "l"(base + s + 16 * ((is_v ? per * rank : 0) + c))
                                 : "memory");
                }
                // the tensor cores read K through the async proxy: each lane waits
                // for its copies and fences before the warp's arrival
                asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            }
            last_q = static_cast<int>(q);
            if constexpr (kFp8) {
                float *const scl = reinterpret_cast<float *>(smem + L::off_scl) + (m & 1) * 3 * kN + lane;
                if (m >= 2 && !(ok = wait_warp(L::scl_free + (m & 1), (m >> 1) - 1))) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!is_v) {
                        scl[32 * i] = s_now[i];
                    } else {
                        // 2^e <= scale < 2^(e+1).  Between 2^-40 and 2^80 the reference follows
                        // it; a smaller one's (values under 4e-10, or zeros) weights fade
                        // below fp16's range, and their sums stay in float32's
                        const int ex = static_cast<int>((__float_as_uint(s_now[i]) >> 23) & 0xffu) - 127;
                        scl[kN + 32 * i] = static_cast<float>(min(max(ex, -40), 80));
                        scl[2 * kN + 32 * i] = s_now[i];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::scl_full + (m & 1)]);
                if (m + 1 < w.ntiles) scales(next, s_now);
            }
            now = next;
        }
        if (!ok) {  // what was copied lands before the memory goes
            const int n_slots = kFp8 ? L::raw : L::slots, step = kFp8 ? 2 : 1;
            for (int k = last_q; k >= 0 && k > last_q - n_slots; k -= step)
                mbar_wait(&bars[(kFp8 || !is_v ? L::k_full : L::v_full) + k % n_slots], (k / n_slots) & 1, nullptr);
        }
    } else if (warp >= kWarpConv && warp < kWarpConv + kConvWarps) {
        // ---------------- conversion to fp16 ----------------
        const int t = tid - kWarpConv * 32;
        bool ok = true;
        if constexpr (!kFp8) {
            for (int n = 0; ok && n < w.ntiles; ++n) {
                const int slot = n % L::slots;
                if (!(ok = wait_warp(L::v_full + slot, n / L::slots))) break;
                uint4 *const v = reinterpret_cast<uint4 *>(smem + L::off_v + slot * kSlotBytes) + t;
#pragma unroll
                for (int i = 0; i < 16; i += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = v[(i + j) * 128];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[(i + j) * 128] = make_uint4(pack_f16(bf16_lo(x[j].x), bf16_hi(x[j].x)), pack_f16(bf16_lo(x[j].y), bf16_hi(x[j].y)),
                                                      pack_f16(bf16_lo(x[j].z), bf16_hi(x[j].z)), pack_f16(bf16_lo(x[j].w), bf16_hi(x[j].w)));
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive_first(&bars[L::v_ready + slot]);
            }
        } else {
            for (int q = 0; ok && q < 2 * w.ntiles; ++q) {
                const int n = q >> 1, slot = n % L::slots, raw = q % L::raw;
                const bool is_v = q & 1;
                if (!(ok = wait_warp(L::k_full + raw, q / L::raw))) break;
                if (n >= L::slots && !(ok = wait_warp((is_v ? L::v_free : L::k_free) + slot, n / L::slots - 1))) break;
                const uint8_t *const src = smem + L::off_raw + raw * kRawBytes;
                uint8_t *const dst = smem + (is_v ? L::off_v : L::off_k) + slot * kSlotBytes;
                // eight lanes take four chunks of 16 codes of rows r and r + 4: both
                // the reads and the writes (one order each for the two rows) then
                // touch every bank once
                const int quads = is_v ? 2 : 4, plane = is_v ? 0 : 8192, region = is_v ? kVRegion : kKRegion;
                const int odd = (t >> 2) & 1;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int u = i * 16 + (t >> 3), p = u / quads, c = 4 * (u - p * quads) + (t & 3);
                    const int r = (p >> 2) * 8 + (p & 3) + 4 * odd;
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + (c >> 3) * plane + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                    uint4 y[2];
                    f16_of_codes(x.x, y[0].x, y[0].y);
                    f16_of_codes(x.y, y[0].z, y[0].w);
                    f16_of_codes(x.z, y[1].x, y[1].y);
                    f16_of_codes(x.w, y[1].z, y[1].w);
                    uint8_t *const to = dst + (c >> 2) * region + r * 128;
                    const int c0 = (2 * c) & 7;
                    *reinterpret_cast<uint4 *>(to + (((c0 + odd) ^ (r & 7)) << 4)) = odd ? y[1] : y[0];
                    *reinterpret_cast<uint4 *>(to + (((c0 + 1 - odd) ^ (r & 7)) << 4)) = odd ? y[0] : y[1];
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[L::raw_free + raw]);
                    arrive_first(&bars[(is_v ? L::v_ready : L::k_ready) + slot]);
                }
            }
        }
    } else if (rank == 0 && lane == 0) {
        // ---------------- products ----------------
        bool ok = true;
        if (warp == kWarpS) {
            const uint32_t idesc = mma_idesc_pair(kN, false, kFp8);
            const uint64_t desc = smem_desc(0, 16, 1024);
            ok = wait_both(L::q_full, 0);
            for (int n = 0; ok && n < w.ntiles; ++n) {
                const int slot = n % L::slots;
                if (n > 0 && !(ok = wait_both(L::s_empty, n - 1))) break;
                if (!kFp8 && !(ok = wait(L::k_full + slot, n / L::slots))) break;
                if (!(ok = wait_both(L::k_ready + slot, n / L::slots))) break;
                tc_fence_after();
                const uint64_t dk = desc + ((sbase + L::off_k + slot * kSlotBytes) >> 4);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    tc_mma_ts_pair(tmem + kSCol, tmem + kQCol + 8 * i, dk + (((i >> 2) * kKRegion + (i & 3) * 32) >> 4), idesc, i > 0);
                tc_commit_pair(&bars[L::k_free + slot]);
                tc_commit_pair(&bars[L::s_full]);
            }
        } else {
            const uint32_t idesc = mma_idesc_pair(kHeadDim, true, true);
            const uint64_t desc_v = smem_desc(0, kVRegion, 1024), desc_p = smem_desc(sbase, 16, 1024);
            for (int n = 0; ok && n < w.ntiles; ++n) {
                const int slot = n % L::slots;
                if (!(ok = wait_both(L::p_full, n))) break;
                if (!(ok = wait_both(L::v_ready + slot, n / L::slots))) break;
                tc_fence_after();
                const uint64_t dv = desc_v + ((sbase + L::off_v + slot * kSlotBytes) >> 4);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    tc_mma_pair(tmem + kOCol, desc_p + (((i >> 2) * kPRegion + (i & 3) * 32) >> 4), dv + (i * 2048 >> 4), idesc,
                                n > 0 || i > 0);
                tc_commit_pair(&bars[L::v_free + slot]);
                tc_commit_pair(&bars[L::o_done]);
            }
        }
        if (!ok) {  // no product is in flight when the tensor memory goes
            const int drain = L::drain + (warp == kWarpPv);
            tc_commit_pair(&bars[drain]);
            mbar_wait(&bars[drain], 0, nullptr);
        }
    } else if (!kFp8 && rank == 1 && warp == kWarpS && lane == 0) {
        // the second CTA's K rows are there
        for (int n = 0; n < w.ntiles; ++n) {
            if (!wait(L::k_full + n % L::slots, n / L::slots)) break;
            fence_async_smem();
            arrive_first(&bars[L::k_ready + n % L::slots]);
        }
    }

    if (tid == 0) pdl_wait();  // the kernel before is done once this grid is
    tc_fence_before();
    cluster_sync();  // both CTAs are done with each other's barriers and products
    if (warp == kWarpS) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Merge of a query row's partials: the shared part's splits, then the pieces of
// the stream's own positions, in that order.  A CTA a row; 64 threads hold its
// 256 dims, and four such groups take every fourth partial and add up at the
// end, so that a row of 40 partials is two rounds of loads.
constexpr int kCombThreads = 256;
constexpr int kCombBatch = 8;

struct CombineArgs {
    const float *ws, *ws_own;
    uint16_t *out;
    int32_t pieces;
    int8_t of[PKV_MAX_SEQS];  // a stream's group, or -1
    PrefixGroup g[kMaxGroups];
};

__global__ void __launch_bounds__(kCombThreads)
    prefix_combine(const __grid_constant__ Common c, const __grid_constant__ CombineArgs a) {
    __shared__ float4 sh[3][64];
    const int tok = blockIdx.x / c.n_q_heads, head = blockIdx.x - tok * c.n_q_heads;
    const int s = find_seq(c.n_seqs, tok, [&](int t) { return c.seq[t].tok_off; });
    const SeqDev &sd = c.seq[s];
    const int kvh = head / c.group, h = head - kvh * c.group;
    const int n_own = sd.nsplit * a.pieces, col = (tok - sd.tok_off) * c.group + h;
    const float *own = a.ws_own + sd.ws_off + ((int64_t)kvh * n_own * sd.ncols + col) * kHeadDim;
    const float *own_ml = a.ws_own + sd.ws_off + (int64_t)c.n_kv_heads * n_own * sd.ncols * kHeadDim + ((int64_t)kvh * n_own * sd.ncols + col) * 2;
    const int64_t own_step = sd.ncols;
    const float *sha = own, *sha_ml = own_ml;
    int n_sha = 0;
    int64_t sha_step = 0;
    if (a.of[s] >= 0) {
        const PrefixGroup &g = a.g[a.of[s]];
        n_sha = g.nsplit;
        sha_step = g.rows;
        const int64_t row = (int64_t)kvh * g.nsplit * g.rows + (tok - g.tok0) * c.group + h;
        sha = a.ws + g.ws_off + row * kHeadDim;
        sha_ml = a.ws + g.ws_off + (int64_t)c.n_kv_heads * g.nsplit * g.rows * kHeadDim + row * 2;
    }
    const int np = n_sha + n_own;
    const int tid = threadIdx.x, lane = tid & 31, grp = tid >> 6, d = 4 * (tid & 63);
    asm volatile("" ::"l"(own), "l"(own_ml), "l"(sha), "l"(sha_ml), "r"(np));
    pdl_wait();
    if (tid == 0) pdl_trigger();  // every kernel of the call but this one is done
    const auto ml_of = [&](int i) -> float2 {
        return __ldcg(reinterpret_cast<const float2 *>(i < n_sha ? sha_ml + 2 * i * sha_step : own_ml + 2 * (i - n_sha) * own_step));
    };
    const auto acc_of = [&](int i) -> float4 {
        return __ldcg(reinterpret_cast<const float4 *>((i < n_sha ? sha + i * sha_step * kHeadDim : own + (i - n_sha) * own_step * kHeadDim) + d));
    };
    const float2 none = make_float2(-INFINITY, 0.f);
    float4 v[kCombBatch];
#pragma unroll
    for (int j = 0; j < kCombBatch; ++j)
        if (grp + 4 * j < np) v[j] = acc_of(grp + 4 * j);
    // every warp finds the row's maximum and sum by itself: lane i has partials i, i + 32, ...
    const float2 ml0 = lane < np ? ml_of(lane) : none, ml1 = lane + 32 < np ? ml_of(lane + 32) : none;
    float M = fmaxf(ml0.x, ml1.x);
    for (int i = lane + 64; i < np; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const auto weight = [&](float m) { return M == -INFINITY ? 0.f : ex2(m - M); };
    const float w0 = weight(ml0.x), w1 = weight(ml1.x);
    float sum = w0 * ml0.y + w1 * ml1.y;
    for (int i = lane + 64; i < np; i += 32) {
        const float2 x = ml_of(i);
        sum += weight(x.x) * x.y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = grp; b < np; b += 4 * kCombBatch) {
        if (b > grp)
#pragma unroll
            for (int j = 0; j < kCombBatch; ++j)
                if (b + 4 * j < np) v[j] = acc_of(b + 4 * j);
#pragma unroll
        for (int j = 0; j < kCombBatch; ++j) {
            const int i = b + 4 * j;
            if (i >= np) break;  // uniform in the warp
            const float w = i < 64 ? __shfl_sync(0xffffffffu, i < 32 ? w0 : w1, i & 31) : weight(ml_of(i).x);
            o4.x = fmaf(w, v[j].x, o4.x);
            o4.y = fmaf(w, v[j].y, o4.y);
            o4.z = fmaf(w, v[j].z, o4.z);
            o4.w = fmaf(w, v[j].w, o4.w);
        }
    }
    if (grp) sh[grp - 1][tid & 63] = o4;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const float4 x = sh[k][tid];
        o4.x += x.x;
        o4.y += x.y;
        o4.z += x.z;
        o4.w += x.w;
    }
    uint2 pk;
    pk.x = pack_bf16(__fdiv_rn(o4.x, sum), __fdiv_rn(o4.y, sum));
    pk.y = pack_bf16(__fdiv_rn(o4.z, sum), __fdiv_rn(o4.w, sum));
    *reinterpret_cast<uint2 *>(a.out + (int64_t)blockIdx.x * kHeadDim + d) = pk;
}

// Split model, in hundredths of a microsecond: a pair's tile of 128 keys and 256
// rows, its start and end, and a split's partials written and read again.
constexpr int64_t kTileCost = 140, kPairCost = 600, kPartialCost = 6;

}  // namespace

// Keys are split into whole tiles, all groups by the same number, so that the
// pairs fill the GPU about once; the count never passes the pairs the GPU holds
// (or one a unit), which bounds the workspace whatever the lengths.
void plan_prefix(const Common &c, int nsm, PrefixPlan *plan) {
    const int64_t H = c.n_kv_heads, slots = std::max(1, nsm / 2);
    int64_t units = 0, most = 1, tile_rows = 0;
    for (int i = 0; i < plan->n_groups; ++i) {
        PrefixGroup &g = plan->group[i];
        const int64_t mtiles = (g.rows + kRows - 1) / kRows;
        units += H * mtiles;
        tile_rows = std::max(tile_rows, (g.rows + mtiles - 1) / mtiles);
        most = std::max<int64_t>(most, ((int64_t)g.len + kN - 1) / kN);
    }
    const auto items_of = [&](int64_t per) {
        int64_t n = 0;
        for (int i = 0; i < plan->n_groups; ++i) {
            const PrefixGroup &g = plan->group[i];
            n += H * ((g.rows + kRows - 1) / kRows) * ((((int64_t)g.len + kN - 1) / kN + per - 1) / per);
        }
        return n;
    };
    const int64_t cap = std::max(units, slots);
    int64_t best = INT64_MAX, chosen = most;
    for (int64_t k = 1; k <= slots; ++k) {
        const int64_t per = (most + k - 1) / k, items = items_of(per);
        if (items > cap) continue;
        const int64_t cost = (items + slots - 1) / slots * (per * kTileCost + kPairCost) + items * kPartialCost;
        if (cost < best) {
            best = cost;
            chosen = per;
        }
    }
    // the most partial rows of `cap` pairs: more than the items' own, which are at
    // most that many of at most tile_rows rows each
    plan->floats = plan->n_groups ? cap * tile_rows * (kHeadDim + 2) + 64 * plan->n_groups : 0;
    int64_t floats = 0;
    plan->items = 0;
    for (int i = 0; i < plan->n_groups; ++i) {
        PrefixGroup &g = plan->group[i];
        const int64_t tiles = std::max<int64_t>(1, ((int64_t)g.len + kN - 1) / kN);
        g.work_off = plan->items;
        g.split_tiles = static_cast<int32_t>(std::min(chosen, tiles));
        g.nsplit = static_cast<int32_t>((tiles + g.split_tiles - 1) / g.split_tiles);
        g.ws_off = floats;
        plan->items += static_cast<int32_t>(H * ((g.rows + kRows - 1) / kRows) * g.nsplit);
        floats += (H * g.nsplit * g.rows * (kHeadDim + 2) + 63) / 64 * 64;
    }
}

int launch_prefix(const Common &c, const PrefixPlan &plan, const DecodeMaps &maps, const uint16_t *q, float *ws,
                  cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    if (once_per_device(attr_done, [] {
            const cudaError_t e = cudaFuncSetAttribute(prefix_partial<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<false>::smem);
            if (e != cudaSuccess) return PKV_ECUDA;
            return cuda_rc(cudaFuncSetAttribute(prefix_partial<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<true>::smem));
        }) != PKV_OK)
        return PKV_ECUDA;
    PrefixArgs a;
    a.q = q;
    a.ws = ws;
    a.status = c.status;
    a.n_groups = plan.n_groups;
    a.n_kv_heads = c.n_kv_heads;
    a.n_q_heads = c.n_q_heads;
    a.group = c.group;
    std::copy(plan.group, plan.group + kMaxGroups, a.g);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * plan.items));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = c.kv_fp8 ? Lay<true>::smem : Lay<false>::smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto *const fn = c.kv_fp8 ? prefix_partial<true> : prefix_partial<false>;
    return launch_status(cudaLaunchKernelEx(&cfg, fn, maps, a));
}

int launch_prefix_combine(const Common &c, const PrefixPlan &plan, int32_t pieces, const float *ws, const float *ws_own,
                          uint16_t *out, cudaStream_t stream) {
    CombineArgs a;
    a.ws = ws;
    a.ws_own = ws_own;
    a.out = out;
    a.pieces = pieces;
    std::copy(plan.of, plan.of + PKV_MAX_SEQS, a.of);
    std::copy(plan.group, plan.group + kMaxGroups, a.g);
    int64_t tokens = 0;
    for (int s = 0; s < c.n_seqs; ++s) tokens += c.seq[s].n_new;
    return launch_status(launch_pdl(prefix_combine, static_cast<unsigned>(tokens * c.n_q_heads), kCombThreads, 0, stream, c, a));
}

}  // namespace pkv
