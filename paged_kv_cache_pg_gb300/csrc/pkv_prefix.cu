// Decode attention over pages that streams share, on the fifth-generation tensor
// cores: the shared rows are read once for all the streams of a group, and every
// stream's own rows in the same pass.
//
// Rows: the query columns of a group's streams on one KV head, token after
// token, 256 to a unit.  Its keys are the shared positions, which every row
// reads, and then the own positions of the streams whose rows these are, stream
// after stream, each of which only its own rows read: counted through as virtual
// keys, in runs of 16, 128 to a tile.  The products of the masked part are idle
// work, a fifth more a tile than a shared one takes; a second kernel for the own
// parts would need partials of its own, and a merge of both.
//
// A pair of CTAs (cta_group::2) takes a unit and a range of its tiles: each CTA
// holds half of the rows, half of a tile's K (64 keys) and half of its V (128
// dims), so a tile's bytes go into shared memory once for 256 rows.  Per tile:
//   S = Q K^T -> TMEM (Q sits there too), P = softmax numerators in fp16 ->
//   shared memory, O += P V -> TMEM
// with V as fp16: bf16 rows are converted where they lie, e4m3 codes (K's too)
// on their way from a raw ring, both exactly (bf16 from 2^-14 on).  So the PV
// product takes one P part of 11 significant bits.  The scales of e4m3 rows go
// into the scores (K) and the weights (V); the weights' reference is the running
// maximum of score + V-scale exponent, so that they stay in fp16's range
// wherever the scales lie.  An own V row that is not finite in fp16 (or lies
// behind its stream's end) is multiplied as zeros, because the other streams'
// rows meet it with a weight of 0; the sums of its stream's rows that read it become
// NaN instead.
//   warps 0-7   softmax: two threads a row, each on 64 of a tile's keys
//   warps 8, 9  copy K and V (halves of one page, of 16-row runs, or key by key)
//   warps 10-13 convert
//   warp 14     first CTA: issues S; second: passes on that its K is there
//   warp 15     first CTA: issues PV
// The splits' O, maxima and sums go to the workspace and prefix_combine merges
// them; a unit of one split writes its output itself.
//
// Of 64 streams on 31,000 shared positions (16 query and 2 KV heads, up to 1,000 own
// positions each; 148 MB, 33.2 GFLOP) a call takes 52.5 us, 632 TFLOP/s: 23 tiles a
// pair of 2,950 cycles, whose 24 products alone take the tensor core 2,620 (16 of N =
// 128 at 96, 8 of N = 256 at 135), 6 us to the first tile, 4.5 for the sums' way out
// and 6 for the merge.  32 streams on 24,000 positions of e4m3 pages take 34.5 us:
// tiles of 3,600 cycles, in which the conversion of 64 KB of codes by four warps is the
// longest chain.
#include <algorithm>
#include <climits>

#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kN = 128;        // keys a tile
constexpr int kRun = 16;       // keys of a run
static_assert(kUnitRows == 2 * kM, "a pair's rows");
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

constexpr int kNear = 1;  // V exponents of a tile this near each other count as their largest
constexpr int kHalfRow = 512, kHalfOut = 256;  // bytes of 128 of a row's float32 sums, of its outputs
constexpr int kMaxSplits = 128;

constexpr int kInfo = 4;  // tiles whose runs' (and scales') places are kept

template <bool kFp8>
struct Lay {
    static constexpr int slots = kFp8 ? 2 : 3;      // of 16-bit K, and of V
    static constexpr int raw = kFp8 ? 3 : 0;        // of codes, K and V in turn
    static constexpr int off_k = 2 * kPRegion;      // P before it
    static constexpr int off_v = off_k + slots * kSlotBytes;
    static constexpr int off_raw = off_v + slots * kSlotBytes;
    static constexpr int off_red = off_raw + raw * kRawBytes;  // [parity][half][row]
    static constexpr int off_scl = off_red + 2 * 2 * kM * 4;   // [tile & 3][K scale, V exponent, V scale][key]
    static constexpr int off_info = off_scl + (kFp8 ? kInfo * 3 * kN * 4 : 0);  // [tile & 3][stream, position, keys][run]
    static constexpr int off_top = off_info + kInfo * 3 * (kN / kRun) * 4;  // [tile & 3]: the largest V exponent
    static constexpr int off_bar = off_top + (kFp8 ? kInfo * 4 : 0);
    // barriers.  Of the first CTA, with arrivals from both: k_ready, v_ready,
    // q_full, s_empty, p_full.  Of each CTA: the others.
    static constexpr int k_full = 0, v_full = 3;      // copies landed (codes: the raw ring's, in k_full)
    static constexpr int raw_free = 6;                // a raw slot is converted
    static constexpr int k_ready = 9, v_ready = 12;   // a slot may be multiplied
    static constexpr int k_free = 15, v_free = 18;    // its products are done
    static constexpr int q_full = 21, s_full = 22, s_empty = 23, p_full = 24, o_done = 25;
    static constexpr int red = 26;                    // a row quarter's exchange (4)
    static constexpr int info_full = 30, info_free = info_full + kInfo;
    static constexpr int drain = info_free + kInfo;
    static constexpr int bars = drain + 2;
    static constexpr int smem = off_bar + bars * 8 + 4 + PKV_MAX_SEQS * 4;  // behind the barriers: TMEM address, positions
    static_assert(smem <= 232448, "above the 227 KB a CTA may hold");
    static_assert(off_k + kSoftWarps * 32 * kHalfRow <= off_red, "the sums fit in the slots");
};

struct PrefixArgs {
    const uint16_t *q;
    uint16_t *out;
    float *ws;
    uint32_t *status;
    int32_t n_units, n_seqs, n_kv_heads, n_q_heads, group;  // group: query heads of a KV head
    alignas(16) int32_t work_off[kMaxUnits];
    PrefixUnit unit[kMaxUnits];
    alignas(16) PrefixStream seq[PKV_MAX_SEQS];
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void arrive_first(uint64_t *bar) {  // at the first CTA's barrier
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(bar, 0)) : "memory");
}
// A bounded wait as mbar_wait, in few instructions where it is called: sixteen
// warps in six roles share the instruction cache, and with each role's loop
// written out at length a tile took 6,500 cycles, half of them waiting for
// instructions.  A role whose wait ran out leaves, and the roles that wait for it,
// in both CTAs, run into the same limit in their turn.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint32_t *status) {
    const uint64_t t0 = global_ns();
    for (uint32_t spin = 1;; ++spin) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((spin & 255u) == 0 && global_ns() - t0 > kWaitLimitNs) {
            if (status) atomicOr(status, PKV_DEV_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, uint32_t *status) {
    return mbar_try_wait(bar, parity) || wait_long(smem_u32(bar), parity, status);
}

// A phase that is known to be over, seen with the cluster's scope.
__device__ __forceinline__ bool mbar_acquired(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// One bulk copy shared -> global (16-byte aligned, whole 16 bytes), and the wait for
// the thread's copies.
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_stores_done() {
    asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// A pair's work.
struct Work {
    int u, kvh, split;
    int first, count;  // the CTA's rows of the unit
    int key0, key1, ntiles;  // virtual keys
};
// The launch parameters that a CTA looks things up in, copied to shared memory
// (where P will be) by all threads at once: read as parameters, each first use of
// a line takes some 600 cycles, one after the other.
struct Stash {
    const PrefixUnit *unit;
    const PrefixStream *seq;
    const int32_t *work_off;
};
__device__ __forceinline__ uint4 load_param16(const void *p) {
    uint4 v;
    asm volatile("ld.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
static_assert(sizeof(PrefixStream) == 24 && PKV_MAX_SEQS % 2 == 0 && sizeof(PrefixUnit) == 128 && kMaxUnits % 4 == 0, "whole 16 bytes");
static_assert(offsetof(PrefixArgs, work_off) % 16 == 0 && offsetof(PrefixArgs, unit) % 16 == 0 && offsetof(PrefixArgs, seq) % 16 == 0 &&
                  alignof(PrefixArgs) >= 16,
              "read 16 bytes at a time");
__device__ __forceinline__ Stash stash_params(const PrefixArgs &a, uint8_t *smem, int tid) {
    const int units = a.n_units * 8, seqs = (a.n_seqs * 24 + 15) / 16, offs = (a.n_units + 3) / 4;
    uint4 *const to = reinterpret_cast<uint4 *>(smem);
    for (int i = tid; i < units + seqs + offs; i += kThreads) {
        const uint8_t *const from = i < units ? reinterpret_cast<const uint8_t *>(a.unit) + 16 * i
                                    : i < units + seqs ? reinterpret_cast<const uint8_t *>(a.seq) + 16 * (i - units)
                                                       : reinterpret_cast<const uint8_t *>(a.work_off) + 16 * (i - units - seqs);
        to[i] = load_param16(from);
    }
    return {reinterpret_cast<const PrefixUnit *>(smem), reinterpret_cast<const PrefixStream *>(to + units),
            reinterpret_cast<const int32_t *>(to + units + seqs)};
}
static_assert(kMaxUnits * 132 + PKV_MAX_SEQS * 24 + 64 <= 2 * kPRegion, "the copies fit where P will be");

__device__ __forceinline__ Work work_of(const Stash &st, int n_units, int item, int rank) {
    Work w;
    w.u = find_seq(n_units, item, [&](int t) { return st.work_off[t]; });
    const PrefixUnit &u = st.unit[w.u];
    const int r = item - st.work_off[w.u], half = (u.rows + 1) >> 1;
    w.kvh = r / u.nsplit;
    w.split = r - w.kvh * u.nsplit;
    w.first = rank * half;
    w.count = rank ? u.rows - half : half;
    const int tiles = (u.keys + kN - 1) / kN, shared = u.shared / kN;
    w.key0 = split_tile(w.split, u.per, shared, tiles) * kN;
    w.key1 = min(u.keys, split_tile(w.split + 1, u.per, shared, tiles) * kN);
    w.ntiles = (w.key1 - w.key0 + kN - 1) / kN;
    return w;
}

// Where a tile's rows are.  With a map: lane i & 7 has run i of 16 rows; without,
// lane i keys i, i + 32, i + 64, i + 96.  Keys behind a stream's end are its last
// one's, runs behind the unit's the tile's first.
struct Look {
    int id[4];      // the page
    int row[4];     // row in it
    int s, pos, n;  // run lane & 7: its stream, its first position, its keys
};

// kRuns: every unit has maps.  The roles share the instruction cache, and code that
// a call does not need costs it: without the copies key by key (16 KB) e4m3 pages of
// 128 took 36.5 us for 38.3, with a loop of its own for the masked tiles' conversion
// and O corrected 16 columns at a time 35.3, with V exponents next to each
// other taken as one 34.6.
template <bool kFp8, bool kRuns>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_partial(const __grid_constant__ DecodeMaps maps, const __grid_constant__ PrefixArgs a) {
    using L = Lay<kFp8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::off_bar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + L::bars);
    int *const bad = reinterpret_cast<int *>(tmem_slot + 1);  // of each stream (from the unit's first): its first V row that is not finite
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
    if (tid == 32 * (kWarpS - 1)) {  // (a warp that copies no parameters below)
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
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(&bars[L::info_full + i], kFp8 ? 2 : 1);
            mbar_init(&bars[L::info_free + i], kSoftWarps + kConvWarps);
        }
        mbar_init(&bars[L::drain], 1);
        mbar_init(&bars[L::drain + 1], 1);
        fence_mbar_init();
    }
    if (warp == kWarpPv) {
        bad[lane] = bad[lane + 32] = INT_MAX;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");  // (the peer lowers them)
    }
    if (warp == kWarpS) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    const Stash stash = stash_params(a, smem, tid);
    tc_fence_before();
    __syncthreads();  // this CTA's barriers, tensor memory and copied parameters are there
    // ... and its peer's, behind this.  Each role goes there once it has read what it
    // needs of the copies, which P's first rows overwrite; the memory's rows, which
    // are the CTA's own, are looked up before
    auto arrive = [&] {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // (the barriers' fence_mbar_init released them)
    };
    auto meet = [&] {
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        tc_fence_after();
    };
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot), sbase = smem_u32(smem);
    const Work w = work_of(stash, a.n_units, static_cast<int>(blockIdx.x >> 1), rank);
    const PrefixUnit &u = a.unit[w.u];
    const PrefixUnit &g = u;  // its group's fields
    const int H = a.n_kv_heads, G = a.group;
    // a tile of shared keys only, none behind their end: nothing to mask
    const auto all_shared = [&](int n) { return w.key0 + (n + 1) * kN <= g.shared; };
    const int *const info = reinterpret_cast<const int *>(smem + L::off_info);  // of tile n: + (n & 3) * 24

    auto wait = [&](int bar, uint32_t phase) -> bool { return wait_on(&bars[bar], phase & 1, a.status); };
    auto wait_warp = [&](int bar, uint32_t phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };
    // The arrivals of the last products at the slots' barriers, which come to both CTAs
    // of the pair whether or not a copy waits for the slot: neither CTA leaves before.
    auto slots_free = [&](int bar) -> bool {
        bool ok = true;
        for (int n = max(0, w.ntiles - L::slots); ok && n < w.ntiles; ++n) ok = wait_warp(bar + n % L::slots, n / L::slots);
        return ok;
    };
    bool settled = false;  // each of the warp's arrivals at the first CTA's barriers has been waited for
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
        int my = -3, qpos = 0;  // the row's stream and position
        int64_t q_row = 0;      // its packed row
        if (row_ok) {
            const PrefixUnit &su = stash.unit[w.u];
            const int gr = su.row0 + w.first + r, t = gr / G, tok = su.tok0 + t, h = gr - t * G;
            my = su.s0 + find_seq(su.n_seqs, tok, [&](int i) { return stash.seq[su.s0 + i].tok; });
            const PrefixStream &st = stash.seq[my];
            qpos = st.len - st.n_new + (tok - st.tok);
            q_row = (int64_t)tok * a.n_q_heads + w.kvh * G + h;
        }
        arrive();
        meet();
        pdl_wait();
        // the next kernel may start: what is older than this grid is done, and
        // this one writes no cached row
        if (tid == 0) pdl_trigger();
        if (active) {
            // Eight lanes read a row's 128 bytes; the rows are turned to their threads
            // where P will be, 64 dims at a time (16 bytes of 32 rows an instruction took
            // 13,600 cycles with 128 e4m3 rows, whose loads miss what is left of L1)
            uint4 v[16];
            const uint4 *const q0 = reinterpret_cast<const uint4 *>(a.q + 128 * hf) + (lane & 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t at = shfl64(row_ok ? q_row : -1, 4 * i + (lane >> 3));
                v[i] = at >= 0 ? __ldg(q0 + at * (kHeadDim / 8)) : make_uint4(0, 0, 0, 0);
                v[8 + i] = at >= 0 ? __ldg(q0 + at * (kHeadDim / 8) + 8) : make_uint4(0, 0, 0, 0);
            }
            uint4 *const turn = reinterpret_cast<uint4 *>(smem) + warp * 256;
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int to = 4 * i + (lane >> 3);
                    turn[8 * to + ((lane & 7) ^ (to & 7))] = v[h + i];
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) v[h + i] = turn[8 * lane + (i ^ (lane & 7))];
                __syncwarp();
            }
            float dn = 1.f;
            if constexpr (kFp8) {
                // bf16 has the wider range: a power of two takes the row's largest
                // element to 2^14 .. 2^15, exactly, and goes into the scores' scale
                uint32_t top = 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                                 __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
                const uint32_t mine = max(top >> 16, top & 0xffffu);
                float other = 0.f;
                ok = exchange(__uint_as_float(mine), other);
                const int ex = static_cast<int>(max(mine, __float_as_uint(other)) >> 7);  // biased exponent
                // (zeros, and rows with an infinity or NaN, stay as they are)
                const int e = ex == 0 || ex == 0xff ? 0 : max(ex - 127 - 14, -100);
                dn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                qs = kScaleLog2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            }
#pragma unroll
            for (int h32 = 0; h32 < 2; ++h32) {
                uint32_t qv[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t e[4] = {v[8 * h32 + i].x, v[8 * h32 + i].y, v[8 * h32 + i].z, v[8 * h32 + i].w};
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
            const int slot = n % kInfo;
            if (!active) {  // no row of the warp: S and P are nobody's
                if (lane == 0) arrive_first(&bars[L::s_empty]);
                if (n > 0 && !(ok = wait_warp(L::o_done, n - 1))) break;
                if (lane == 0) {
                    arrive_first(&bars[L::p_full]);
                    mbar_arrive(&bars[L::info_free + slot]);
                }
                __syncwarp();
                continue;
            }
            const bool masked = !all_shared(n);
            const float *const scl = reinterpret_cast<const float *>(smem + L::off_scl) + slot * 3 * kN + 64 * hf;
            // (S is read before anything else is looked at: the next S product waits for it)
            float x[64];
            tc_fence_after();
            {
                uint32_t sv[64];
                tmem_ld64(lane_base + kSCol + 64 * hf, sv);
#pragma unroll
                for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(sv[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && n + 1 < w.ntiles) arrive_first(&bars[L::s_empty]);
            if ((kFp8 || masked) && !(ok = wait_warp(L::info_full + slot, n / kInfo))) break;
            // the keys that the row sees, a bit each: of a run of its own stream those up
            // to its position, of a shared run those there are
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            bool any = true;
            if (masked) {
                const int4 *const run = reinterpret_cast<const int4 *>(info + slot * 24) + hf;
                const int4 s4 = run[0], p4 = run[2], n4 = run[4];  // streams, positions, keys of the half's four runs
                const auto bits = [&](int st, int pos, int keys) -> uint32_t {
                    const int k = min(keys, st == -1 ? kRun : st == my ? qpos - pos + 1 : 0);
                    return k > 0 ? (1u << k) - 1u : 0u;
                };
                see[0] = bits(s4.x, p4.x, n4.x) | (bits(s4.y, p4.y, n4.y) << 16);
                see[1] = bits(s4.z, p4.z, n4.z) | (bits(s4.w, p4.w, n4.w) << 16);
                any = __any_sync(0xffffffffu, (see[0] | see[1]) != 0u);
            }
            if (kFp8 && any) {
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 k = *reinterpret_cast<const float4 *>(scl + j);
                    const float2 lo = mul2(make_float2(x[j], x[j + 1]), make_float2(k.x, k.y));
                    const float2 hi = mul2(make_float2(x[j + 2], x[j + 3]), make_float2(k.z, k.w));
                    x[j] = lo.x;
                    x[j + 1] = lo.y;
                    x[j + 2] = hi.x;
                    x[j + 3] = hi.y;
                }
            }
            if (masked && any) {
#pragma unroll
                for (int j = 0; j < 64; ++j)
                    if (!(see[j >> 5] & (1u << (j & 31)))) x[j] = -INFINITY;
            }
            // this half's reference as eight interleaved chains, then the row's.  V
            // exponents next to each other (a tile's mostly are) count as the larger: one of
            // fp16's binades, for a third of the scales' reads
            const float2 qs2 = make_float2(qs, qs);
            float m8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) m8[j] = -INFINITY;
            const float top = kFp8 ? reinterpret_cast<const float *>(smem + L::off_top)[slot] : 0.f;
            if (!any) {
            } else if (kFp8 && top == INFINITY) {
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 e = *reinterpret_cast<const float4 *>(scl + kN + j);
                    const float2 lo = fma2(make_float2(x[j], x[j + 1]), qs2, make_float2(e.x, e.y));
                    const float2 hi = fma2(make_float2(x[j + 2], x[j + 3]), qs2, make_float2(e.z, e.w));
                    m8[j & 7] = fmaxf(m8[j & 7], lo.x);
                    m8[(j + 1) & 7] = fmaxf(m8[(j + 1) & 7], lo.y);
                    m8[(j + 2) & 7] = fmaxf(m8[(j + 2) & 7], hi.x);
                    m8[(j + 3) & 7] = fmaxf(m8[(j + 3) & 7], hi.y);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) m8[j & 7] = fmaxf(m8[j & 7], x[j]);
            }
            float lmx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
            if (kFp8 && top != INFINITY) lmx = fmaf(lmx, qs, top);
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
                for (int ch = 0; ch < 8; ++ch) {
                    uint32_t o[16];
                    tmem_ld16(lane_base + kOCol + 128 * hf + ch * 16, o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                    tmem_st16(lane_base + kOCol + 128 * hf + ch * 16, o);
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
            if (!any) {
#pragma unroll
                for (int j = 0; j < 32; ++j) p16[j] = 0u;
            } else if constexpr (kFp8) {
                const float2 off = make_float2(-m_off, -m_off);
                float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(scl + 2 * kN + j);
                    float2 lo = fma2(make_float2(x[j], x[j + 1]), qs2, off), hi = fma2(make_float2(x[j + 2], x[j + 3]), qs2, off);
                    lo.x = ex2(lo.x);
                    lo.y = ex2(lo.y);
                    hi.x = ex2(hi.x);
                    hi.y = ex2(hi.y);
                    ps[0] = add2(ps[0], lo);
                    ps[1] = add2(ps[1], hi);
                    lo = mul2(lo, make_float2(v.x, v.y));
                    hi = mul2(hi, make_float2(v.z, v.w));
                    p16[j / 2] = pack_f16(lo.x, lo.y);
                    p16[j / 2 + 1] = pack_f16(hi.x, hi.y);
                }
                l += (ps[0].x + ps[1].x) + (ps[0].y + ps[1].y);
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::info_free + slot]);
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
        // The last products' arrival comes to both CTAs: warps without rows wait for it
        // too, so that a CTA that has none is still there when it does
        ok = ok && wait_warp(L::o_done, w.ntiles - 1);
        // ---------------- the split's sums to the workspace ----------------
        if (ok && active) {
            float other = 0.f;
            ok = exchange(l, other);
            l += other;
            // (and what the peer's converters flagged before those products)
            ok = ok && mbar_acquired(&bars[L::o_done], (w.ntiles - 1) & 1);
            tc_fence_after();
        }
        if (ok && active) {
            // Through the slots, whose products are done, and out by bulk copies: 16
            // bytes a lane at a time straight from the registers took 3,000 cycles.
            // A split's partials are [32 dims][row][32], a row's 16-byte chunks exchanged
            // by its number's low bits (no two of eight lanes in one bank), so that 32 dims
            // of a warp's 32 rows go as one copy while the next ones are read; a unit's
            // outputs are a copy a lane, its rows 16 bytes apart.
            const bool single = u.nsplit == 1;
            const int wr = 32 * (warp & 3), key = (w.first + r) & 7;
            uint8_t *const stage = smem + L::off_k + warp * 32 * kHalfRow, *const mine = stage + lane * (single ? kHalfOut + 16 : 128);
            // (a new token does not read its stream's later ones)
            const bool odd_row = row_ok && reinterpret_cast<volatile int *>(bad)[my - u.s_first] <= qpos;
            if (odd_row) l = __uint_as_float(0x7fffffffu);
            const float inv = 1.f / l;
            const int64_t split = (int64_t)w.kvh * u.nsplit + w.split;
            float *const acc = a.ws + u.ws_off + split * u.rows * kHeadDim + (int64_t)hf * u.rows * (kHeadDim / 2) + (w.first + wr) * 32;
            float *const ml = a.ws + u.ws_off + (int64_t)H * u.nsplit * u.rows * kHeadDim + split * u.rows * 2;
            float2 odd = make_float2(0.f, 0.f);  // NaN once a sum is not finite
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(lane_base + kOCol + 128 * hf + 32 * ch, o);
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    odd = fma2(make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), make_float2(0.f, 0.f), odd);
                if (single) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t e[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            e[k] = pack_bf16(__uint_as_float(o[8 * j + 2 * k]) * inv, __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
                        *reinterpret_cast<uint4 *>(mine + 16 * (4 * ch + j)) = make_uint4(e[0], e[1], e[2], e[3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4 *>(mine + 4096 * ch + 16 * (j ^ key)) =
                            make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) bulk_s2g(acc + (int64_t)ch * u.rows * 32, stage + 4096 * ch, min(32, w.count - wr) * 128);
                }
            }
            if (single && row_ok) {
                fence_async_smem();
                bulk_s2g(a.out + q_row * kHeadDim + 128 * hf, mine, kHalfOut);
            }
            if (row_ok) {
                if (hf == 0 && !single) *reinterpret_cast<float2 *>(ml + 2 * (w.first + r)) = make_float2(m_used, l);
                if ((odd_row || odd.x + odd.y != 0.f || (m_used != -INFINITY && fabsf(m_used) > kFarScore)) && a.status)
                    atomicOr(a.status, PKV_DEV_RANGE);
            }
            bulk_stores_done();
            settled = true;
        }
        if (!ok && rank == 1 && warp == 0 && lane == 0) {  // (the first CTA's issuers gave up, or soon will)
            wait_on(&bars[L::drain], 0, nullptr);
            wait_on(&bars[L::drain + 1], 0, nullptr);
        }
    } else if (warp == kWarpK || warp == kWarpV) {
        // ---------------- copies ----------------
        const bool is_v = warp == kWarpV;
        const PrefixUnit &su = stash.unit[w.u];
        const int ptok = su.ptok, n_pages = su.n_pages, shared = su.shared, keys = su.keys, s_first = su.s_first;
        const int64_t page_elems = su.ps;
        const uint64_t pol = policy_evict_normal();  // other units read the shared rows too
        const void *const map = kRuns || su.map_run >= 0 ? &maps.map[su.map_run] : nullptr;
        const int whole_map = is_v ? su.map_v : su.map_k;
        const void *const map_w = whole_map >= 0 ? &maps.map[whole_map] : nullptr;
        const uint8_t *const base = reinterpret_cast<const uint8_t *>(su.layer_base);
        const bool runs = kRuns || map != nullptr;
        if (runs && lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
            if (map_w) asm volatile("prefetch.tensormap [%0];" ::"l"(map_w) : "memory");
        }
        // The unit's streams, one and another 32 behind it a lane: a search through
        // the launch parameters for each run took a tile of 64 streams 3 us
        const int pad = (shared + kRun - 1) / kRun * kRun, n_seqs = su.s0 + su.n_seqs - s_first;
        int st_own[2], st_len[2];
        int64_t st_table[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = min(lane + 32 * i, n_seqs - 1);
            const PrefixStream &st = stash.seq[s_first + t];
            st_own[i] = lane + 32 * i < n_seqs ? st.own : INT_MAX;
            st_len[i] = st.len;
            st_table[i] = reinterpret_cast<int64_t>(st.table);
        }
        const int layer_row = static_cast<int>(su.layer_row), early = min(shared, su.early);
        arrive();
        const int own0 = __shfl_sync(0xffffffffu, st_own[0], 0);
        const int64_t table0 = shfl64(st_table[0], 0);  // (every lane takes part in every exchange: none under a lane's condition)
        auto look = [&](int m) -> Look {
            Look k;
            const int kt = w.key0 + m * kN, v = kt + kRun * (lane & 7);
            // run lane & 7: the last stream whose own keys begin at or before its first
            int t = 0;
            if (kt + kN > pad) {  // uniform
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const int x = kt + kRun * i - pad + own0;
                    const int below = __popc(__ballot_sync(0xffffffffu, st_own[0] <= x)) + __popc(__ballot_sync(0xffffffffu, st_own[1] <= x));
                    if ((lane & 7) == i) t = max(below - 1, 0);
                }
            }
            const auto pick = [&](int x, int y) {
                const int lo = __shfl_sync(0xffffffffu, x, t & 31), hi = __shfl_sync(0xffffffffu, y, t & 31);
                return t < 32 ? lo : hi;
            };
            const int own = pick(st_own[0], st_own[1]), len = pick(st_len[0], st_len[1]);
            const int64_t table_lo = shfl64(st_table[0], t & 31), table_hi = shfl64(st_table[1], t & 31);
            const int64_t table = v < pad ? table0 : t < 32 ? table_lo : table_hi;
            const int limit = v < pad ? shared : len;
            k.s = v >= keys ? -2 : v < pad ? -1 : s_first + t;
            k.pos = v < pad ? v : shared + (v - pad + own0 - own);
            k.n = k.s == -2 ? 0 : min(kRun, limit - k.pos);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                k.id[i] = 0;
                k.row[i] = 0;
                if (runs && i > 0) continue;
                // the key's run (behind the unit's last one: the tile's first), from its lane
                int src = runs ? lane & 7 : 2 * i + (lane >> 4);
                if (__shfl_sync(0xffffffffu, k.s, src) == -2) src = 0;
                const int first = __shfl_sync(0xffffffffu, k.pos, src), last = __shfl_sync(0xffffffffu, limit, src) - 1;
                const int32_t *const tab = reinterpret_cast<const int32_t *>(shfl64(table, src));
                const int pos = runs ? first : min(first + (lane & 15), last);
                const int page = tab ? pos / ptok : 0;
                k.row[i] = pos - page * ptok;
                k.id[i] = tab ? __ldg(tab + page) : 0;  // (not looked at before its tile's turn)
            }
            return k;
        };
        // element offset of a looked-up page from layer_base; one outside the arena is
        // reported and read as page 0
        auto page_at = [&](int id) -> int64_t {
            if (static_cast<uint32_t>(id) < static_cast<uint32_t>(n_pages)) return (int64_t)id * page_elems;
            if (!is_v && a.status) atomicOr(a.status, PKV_DEV_BAD_PAGE);
            return 0;
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
                    at = page_at(__shfl_sync(0xffffffffu, k.id[0], src));
                    row = __shfl_sync(0xffffffffu, k.row[0], src) + (lane & 15);
                } else {
                    at = page_at(k.id[i]);
                    row = k.row[i];
                }
                s[i] = __ldg(reinterpret_cast<const float *>(base + 2 * at + off8_scale(is_v, H, ptok, w.kvh, row)));
            }
        };
        float s_now[4] = {0.f, 0.f, 0.f, 0.f};
        // Shared positions far enough below the new tokens stream before the kernel
        // before this one is done (it may be storing this call's new rows)
        bool waited = false;
        int last_q = -1;
        bool ok = true;
        // Key by key, a bf16 tile's copies are on their way while the next one's are
        // issued, and it is told of after that (45 streams on 6,168 positions, pages of
        // 4: 68.4 us for 73.2; the codes' three slots are too few: 28.5 for 26.8 there).
        // The tensor cores read K through the async proxy: each lane waits for its
        // copies and fences before the warp's arrival.
        uint64_t *held = nullptr;
        auto landed = [&] {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(held);
            held = nullptr;
        };
        for (int m = 0; ok && m < w.ntiles; ++m) {
            // looked up while the slot is still being multiplied
            const Look now = look(m);
            if (!waited && w.key0 + (m + 1) * kN > early) {
                pdl_wait();
                waited = true;
            }
            if constexpr (kFp8) scales(now, s_now);
            if (m == 0) meet();
            // the slot
            const uint32_t q = kFp8 ? 2 * m + is_v : m;
            const uint32_t n_slots = kFp8 ? L::raw : L::slots, slot = q % n_slots;
            if (q >= n_slots) {
                const int free = (kFp8 ? L::raw_free : is_v ? L::v_free : L::k_free) + slot;
                const uint32_t phase = q / n_slots - 1;
                // (nothing is held back from those who would free it)
                if (held && !__all_sync(0xffffffffu, mbar_acquired(&bars[free], phase & 1))) {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    landed();
                }
                if (!(ok = wait_warp(free, phase))) break;
            }
            uint64_t *const full = &bars[(kFp8 || !is_v ? L::k_full : L::v_full) + slot];
            uint8_t *const dst = smem + (kFp8 ? L::off_raw + slot * kRawBytes : (is_v ? L::off_v : L::off_k) + slot * kSlotBytes);
            if (runs) {
                const int64_t rb = row_bytes(page_at(now.id[0]), now.row[0]);
                const int y = layer_row + static_cast<int>(rb / (kFp8 ? 256 : 512));
                if (lane == 0) mbar_arrive_expect_tx(full, kFp8 ? kRawBytes : kSlotBytes);
                __syncwarp();  // the expected bytes come first
                // K's 64 keys, or V's 128, row after row in memory (one page's, mostly)
                const int run0 = is_v ? 0 : 4 * rank, n_runs = is_v ? 8 : 4;
                const int yf = __shfl_sync(0xffffffffu, y, run0);
                const bool in_row = (lane & 7) < run0 || (lane & 7) >= run0 + n_runs || y == yf + 16 * ((lane & 7) - run0);
                if (map_w && __all_sync(0xffffffffu, in_row)) {
                    // one copy (two of K's code halves)
                    if (kFp8) {
                        if (lane < (is_v ? 1 : 2))
                            tma_load_2d(dst + lane * 8192, map_w, is_v ? 128 * rank : 128 * lane, yf, full, pol);
                    } else if (lane == 0) {
                        tma_load_3d(dst, map_w, 0, yf, is_v ? 2 * rank : 0, full, pol);
                    }
                } else {
                    // 16-row runs, one box a lane: K four runs of all dims, V eight of half
                    const int nc = kFp8 ? (is_v ? 1 : 2) : (is_v ? 2 : 4);  // boxes of a run
                    const int rn = lane / nc, ch = lane - rn * nc;
                    const int yr = __shfl_sync(0xffffffffu, y, (run0 + rn) & 7);
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
                // key by key: 16-byte chunks through the same swizzle, the row's place by one
                // exchange (four, with the selects behind them, took a tile 3 us longer)
                int64_t src[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) src[i] = row_bytes(page_at(now.id[i]), now.row[i]);
                constexpr int kChunks = kFp8 ? 16 : 32;  // of a row
                const int per = is_v ? kChunks / 2 : kChunks, rows_pass = 32 / per, n_groups = is_v ? 4 : 2;
                const int c = lane % per, sub = lane / per;
                const int region = is_v ? 128 * 128 : 64 * 128;
                const uint8_t *const chunk = base + 16 * ((is_v ? per * rank : 0) + c);
#pragma unroll 1
                for (int g = 0; g < n_groups; ++g) {
                    // the group's 32 keys are src[at]'s (by selects: an index would put them in memory)
                    const int at = is_v ? g : 2 * rank + g;
                    const int64_t mine = at == 0 ? src[0] : at == 1 ? src[1] : at == 2 ? src[2] : src[3];
                    uint8_t *const to = dst + (c >> 3) * region + 32 * g * 128;
#pragma unroll 4
                    for (int r0 = 0; r0 < 32; r0 += rows_pass) {
                        const int r = r0 + sub;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         smem_u32(to + r * 128 + (((c & 7) ^ (r & 7)) << 4))),
                                     "l"(chunk + shfl64(mine, r))
                                     : "memory");
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (!kFp8 && held) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    landed();
                }
                held = full;
                if (kFp8) {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    landed();
                }
            }
            last_q = static_cast<int>(q);
            // the runs' places, and with e4m3 the scales
            if (kFp8 || !is_v) {
                const int is = m % kInfo;
                if (m >= kInfo && !(ok = wait_warp(L::info_free + is, m / kInfo - 1))) break;
                if (!is_v && lane < 8) {
                    int *const to = reinterpret_cast<int *>(smem + L::off_info) + is * 24 + lane;
                    to[0] = now.s;
                    to[8] = now.pos;
                    to[16] = now.n;
                }
                if constexpr (kFp8) {
                    float *const scl = reinterpret_cast<float *>(smem + L::off_scl) + is * 3 * kN + lane;
                    int most = -127, least = 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!is_v) {
                            scl[32 * i] = s_now[i];
                        } else {
                            // Other streams' rows meet an own row with a weight of 0, which a
                            // scale that is not finite must not make NaN: it counts as 0, and
                            // its place is kept.  Behind the run's keys it may be anything.
                            const int run = 2 * i + (lane >> 4);
                            const int st = __shfl_sync(0xffffffffu, now.s, run), n = __shfl_sync(0xffffffffu, now.n, run);
                            const int pos = __shfl_sync(0xffffffffu, now.pos, run) + (lane & 15);
                            if ((lane & 15) >= n) {
                                s_now[i] = 0.f;
                            } else if (st >= 0 && !(fabsf(s_now[i]) < INFINITY)) {
                                s_now[i] = 0.f;
                                atomicMin(bad + (st - s_first), pos);
                            }
                            // 2^e <= scale < 2^(e+1).  Between 2^-40 and 2^80 the reference follows
                            // it; a smaller one's (values under 4e-10, or zeros) weights fade
                            // below fp16's range, and their sums stay in float32's
                            const int ex = static_cast<int>((__float_as_uint(s_now[i]) >> 23) & 0xffu) - 127;
                            const int e = min(max(ex, -40), 80);
                            scl[kN + 32 * i] = static_cast<float>(e);
                            scl[2 * kN + 32 * i] = s_now[i];
                            most = max(most, e);
                            least = min(least, e);
                        }
                    }
                    if (is_v) {
                        most = __reduce_max_sync(0xffffffffu, most);
                        least = __reduce_min_sync(0xffffffffu, least);
                        if (lane == 0)
                            reinterpret_cast<float *>(smem + L::off_top)[is] = most - least <= kNear ? static_cast<float>(most) : INFINITY;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::info_full + is]);
            }
        }
        if (held) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            landed();
        }
        if constexpr (!kFp8) ok = ok && slots_free(is_v ? L::v_free : L::k_free);
        if (!ok) {  // what was copied lands before the memory goes
            const int n_slots = kFp8 ? L::raw : L::slots, step = kFp8 ? 2 : 1;
            for (int k = last_q; k >= 0 && k > last_q - n_slots; k -= step)
                mbar_wait(&bars[(kFp8 || !is_v ? L::k_full : L::v_full) + k % n_slots], (k / n_slots) & 1, nullptr);
        }
    } else if (warp >= kWarpConv && warp < kWarpConv + kConvWarps) {
        // ---------------- conversion to fp16 ----------------
        arrive();
        meet();
        const int t = tid - kWarpConv * 32;
        bool ok = true;
        const auto flag = [&](int s, int pos) {  // in both CTAs: each converts half of the dims
            for (uint32_t r = 0; r < 2; ++r)
                asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(peer_addr(bad + (s - u.s_first), r)), "r"(pos)
                             : "memory");
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
        };
        // Of a tile that is not all shared: bit i is set where row `row` of run i is
        // behind its stream's end
        const auto behind = [&](const int *run, int row) -> uint32_t {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) m |= (row >= run[16 + i] ? 1u : 0u) << i;
            return m;
        };
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        // of eight fp16 values, the largest magnitudes' bits of the four low and the four
        // high halves
        const auto largest = [](const uint4 &v) {
            return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        };
        const auto not_finite = [](uint32_t m) { return (m & 0xffffu) >= 0x7c00u || (m >> 16) >= 0x7c00u; };
        if constexpr (!kFp8) {
            for (int n = 0; ok && n < w.ntiles; ++n) {
                const int slot = n % L::slots;
                if (!(ok = wait_warp(L::v_full + slot, n / L::slots))) break;
                uint4 *const v = reinterpret_cast<uint4 *>(smem + L::off_v + slot * kSlotBytes) + t;
                const bool masked = !all_shared(n);
                if (masked && !(ok = wait_warp(L::info_full + n % kInfo, n / kInfo))) break;
                const int *const run = info + n % kInfo * 24;  // chunk i of a thread lies in run i & 7, row t >> 3
                const uint32_t none = masked ? behind(run, t >> 3) : 0u;
                uint32_t top = 0u;  // the largest magnitude's bits
#pragma unroll 1
                for (int i = 0; i < 16; i += 4) {
                    uint4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = v[(i + j) * 128];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (none & (1u << ((i + j) & 7))) x[j] = zero;
                        const uint4 y = make_uint4(pack_f16(bf16_lo(x[j].x), bf16_hi(x[j].x)), pack_f16(bf16_lo(x[j].y), bf16_hi(x[j].y)),
                                                   pack_f16(bf16_lo(x[j].z), bf16_hi(x[j].z)), pack_f16(bf16_lo(x[j].w), bf16_hi(x[j].w)));
                        if (masked) top = __vmaxu2(top, largest(y));
                        v[(i + j) * 128] = y;
                    }
                }
                if (masked && not_finite(top)) {
                    // something is not finite: chunks of own rows that have it become zeros
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        if (run[i & 7] >= 0 && not_finite(largest(v[i * 128]))) {
                            v[i * 128] = zero;
                            flag(run[i & 7], run[8 + (i & 7)] + (t >> 3));
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    // (first: a softmax warp's arrival for a later tile comes behind v_ready's)
                    mbar_arrive(&bars[L::info_free + n % kInfo]);
                    arrive_first(&bars[L::v_ready + slot]);
                }
            }
        } else {
            // Eight lanes take four chunks of 16 codes of rows r and r + 4: both the reads
            // and the writes (one order each for the two rows) then touch every bank
            // once.  A thread's chunks are the same one of every 8th (K) or 16th (V) row.
            const int odd = (t >> 2) & 1;
            for (int q = 0; ok && q < 2 * w.ntiles; ++q) {
                const int n = q >> 1, slot = n % L::slots, raw = q % L::raw;
                const bool is_v = q & 1;
                if (!(ok = wait_warp(L::k_full + raw, q / L::raw))) break;
                if (n >= L::slots && !(ok = wait_warp((is_v ? L::v_free : L::k_free) + slot, n / L::slots - 1))) break;
                const bool masked = is_v && !all_shared(n);
                if (masked && !(ok = wait_warp(L::info_full + n % kInfo, n / kInfo))) break;
                const int *const run = info + n % kInfo * 24;  // V: a thread's chunk i lies in run i
                const int c = 4 * ((t >> 3) & (is_v ? 1 : 3)) + (t & 3), c0 = (2 * c) & 7;
                const int r = (is_v ? ((t >> 6) << 3) + ((t >> 4) & 3) : t >> 5) + 4 * odd, step = is_v ? 2048 : 1024;
                const uint8_t *const src = smem + L::off_raw + raw * kRawBytes + (c >> 3) * 8192 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                uint8_t *const dst = smem + (is_v ? L::off_v + (c >> 2) * kVRegion : L::off_k + (c >> 2) * kKRegion) + slot * kSlotBytes + r * 128;
                uint8_t *const to0 = dst + (((c0 + odd) ^ (r & 7)) << 4), *const to1 = dst + (((c0 + 1 - odd) ^ (r & 7)) << 4);
                const uint32_t none = masked ? behind(run, r) : 0u;
                uint32_t top = 0u;  // the largest magnitude's bits
                if (!masked) {
#pragma unroll 1
                    for (int i = 0; i < 8; i += 4) {
                        uint4 x[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint4 *>(src + (i + j) * step);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint4 y0, y1;
                            f16_of_codes(x[j].x, y0.x, y0.y);
                            f16_of_codes(x[j].y, y0.z, y0.w);
                            f16_of_codes(x[j].z, y1.x, y1.y);
                            f16_of_codes(x[j].w, y1.z, y1.w);
                            *reinterpret_cast<uint4 *>(to0 + (i + j) * step) = odd ? y1 : y0;
                            *reinterpret_cast<uint4 *>(to1 + (i + j) * step) = odd ? y0 : y1;
                        }
                    }
                } else {  // in a loop of its own, so that the first one is small
#pragma unroll 1
                    for (int i = 0; i < 8; i += 2) {
                        uint4 x[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) x[j] = *reinterpret_cast<const uint4 *>(src + (i + j) * step);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (none & (1u << (i + j))) x[j] = zero;
                            uint4 y0, y1;
                            f16_of_codes(x[j].x, y0.x, y0.y);
                            f16_of_codes(x[j].y, y0.z, y0.w);
                            f16_of_codes(x[j].z, y1.x, y1.y);
                            f16_of_codes(x[j].w, y1.z, y1.w);
                            top = __vmaxu2(top, __vmaxu2(largest(y0), largest(y1)));
                            *reinterpret_cast<uint4 *>(to0 + (i + j) * step) = odd ? y1 : y0;
                            *reinterpret_cast<uint4 *>(to1 + (i + j) * step) = odd ? y0 : y1;
                        }
                    }
                }
                if (masked && not_finite(top)) {
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        uint4 *const y0 = reinterpret_cast<uint4 *>(to0 + i * step), *const y1 = reinterpret_cast<uint4 *>(to1 + i * step);
                        if (run[i] >= 0 && not_finite(__vmaxu2(largest(*y0), largest(*y1)))) {
                            *y0 = *y1 = zero;
                            flag(run[i], run[8 + i] + r);
                        }
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[L::raw_free + raw]);
                    if (is_v) mbar_arrive(&bars[L::info_free + n % kInfo]);
                    arrive_first(&bars[(is_v ? L::v_ready : L::k_ready) + slot]);
                }
            }
            if (ok && warp == kWarpConv && slots_free(L::k_free)) slots_free(L::v_free);
        }
    } else {
        arrive();
        meet();
    }
    if (warp >= kWarpS && rank == 0 && lane == 0) {
        // ---------------- products ----------------
        bool ok = true;
        if (warp == kWarpS) {
            const uint32_t idesc = mma_idesc_pair(kN, false, kFp8);
            const uint64_t desc = smem_desc(0, 16, 1024);
            ok = wait(L::q_full, 0);
            for (int n = 0; ok && n < w.ntiles; ++n) {
                const int slot = n % L::slots;
                if (n > 0 && !(ok = wait(L::s_empty, n - 1))) break;
                if (!kFp8 && !(ok = wait(L::k_full + slot, n / L::slots))) break;
                if (!(ok = wait(L::k_ready + slot, n / L::slots))) break;
                tc_fence_after();
                const uint64_t dk = desc + ((sbase + L::off_k + slot * kSlotBytes) >> 4);
#pragma unroll 1
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc_mma_ts_pair(tmem + kSCol, tmem + kQCol + 32 * i + 8 * j, dk + ((i * kKRegion + j * 32) >> 4), idesc, i + j > 0);
                tc_commit_pair(&bars[L::k_free + slot]);
                tc_commit_pair(&bars[L::s_full]);
            }
        } else {
            const uint32_t idesc = mma_idesc_pair(kHeadDim, true, true);
            const uint64_t desc_v = smem_desc(0, kVRegion, 1024), desc_p = smem_desc(sbase, 16, 1024);
            for (int n = 0; ok && n < w.ntiles; ++n) {
                const int slot = n % L::slots;
                if (!(ok = wait(L::p_full, n))) break;
                if (!(ok = wait(L::v_ready + slot, n / L::slots))) break;
                tc_fence_after();
                const uint64_t dv = desc_v + ((sbase + L::off_v + slot * kSlotBytes) >> 4);
#pragma unroll 1
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc_mma_pair(tmem + kOCol, desc_p + ((i * kPRegion + j * 32) >> 4), dv + ((4 * i + j) * 2048 >> 4), idesc,
                                    n + i + j > 0);
                tc_commit_pair(&bars[L::v_free + slot]);
                tc_commit_pair(&bars[L::o_done]);
            }
        }
        if (!ok) {  // no product is in flight when the tensor memory goes
            const int drain = L::drain + (warp == kWarpPv);
            tc_commit_pair(&bars[drain]);
            mbar_wait(&bars[drain], 0, nullptr);
        }
    }
    if (!kFp8 && rank == 1 && warp == kWarpS && lane == 0) {
        // the second CTA's K rows are there
        for (int n = 0; n < w.ntiles; ++n) {
            if (!wait(L::k_full + n % L::slots, n / L::slots)) break;
            fence_async_smem();
            arrive_first(&bars[L::k_ready + n % L::slots]);
        }
    }

    tc_fence_before();
    // both CTAs are done with each other's barriers and products (a warp that has
    // settled has nothing to release but its sums, which the kernel's end does)
    __syncwarp();
    if (settled)
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    else
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (warp == kWarpS) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// Merge of a query row's splits, in their order.  A CTA a row; 64 threads hold
// its 256 dims, and four such groups (two, where the GPU does not hold four of all
// rows at once) take every fourth (second) split and add up at the end.
constexpr int kCombThreads = 256;
constexpr int kCombCtas = 4;  // of kCombThreads an SM holds
constexpr int kCombBatch = 8;

struct CombineArgs {
    const float *ws;
    uint16_t *out;
    int32_t n_groups, n_kv_heads, n_q_heads, group;
    int32_t tok0[PKV_MAX_SEQS];   // of each group
    int32_t unit0[PKV_MAX_SEQS];
    struct Unit {
        int64_t ws_off;
        int32_t rows, nsplit;
    } unit[kMaxUnits];
};

__global__ void __launch_bounds__(kCombThreads, kCombCtas)
    prefix_combine(const __grid_constant__ CombineArgs a) {
    __shared__ float weight[kMaxSplits];
    __shared__ float4 sh[3][64];
    const int tok = blockIdx.x / a.n_q_heads, head = blockIdx.x - tok * a.n_q_heads;
    const int k = find_seq(a.n_groups, tok, [&](int t) { return a.tok0[t]; });
    const int kvh = head / a.group, row = (tok - a.tok0[k]) * a.group + head - kvh * a.group;
    const CombineArgs::Unit &u = a.unit[a.unit0[k] + row / kUnitRows];
    const int np = u.nsplit, groups = blockDim.x >> 6;
    const int64_t first = (int64_t)kvh * np * u.rows;
    const int tid = threadIdx.x, lane = tid & 31, grp = tid >> 6, ur = row % kUnitRows;
    const int step = u.rows * kHeadDim;
    const float *const acc = a.ws + u.ws_off + first * kHeadDim + (((tid & 63) >> 3) * u.rows + ur) * 32 + 4 * ((tid ^ ur) & 7);
    const float2 *const ml = reinterpret_cast<const float2 *>(a.ws + u.ws_off + (int64_t)a.n_kv_heads * np * u.rows * kHeadDim) + first + ur;
    asm volatile("" ::"l"(acc), "l"(ml), "r"(np));
    pdl_wait();
    if (tid == 0) pdl_trigger();
    if (np == 1) return;  // written where it was summed
    float4 v[kCombBatch];
    const auto load = [&](int b) {
#pragma unroll
        for (int j = 0; j < kCombBatch; ++j)
            if (b + groups * j < np) v[j] = __ldcg(reinterpret_cast<const float4 *>(acc + (int64_t)(b + groups * j) * step));
    };
    load(grp);
    // every warp finds the row's maximum and sum by itself: lane i has splits i, i + 32, ...
    float2 x[kMaxSplits / 32];
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxSplits / 32; ++j) {
        x[j] = lane + 32 * j < np ? __ldcg(ml + (int64_t)(lane + 32 * j) * u.rows) : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, x[j].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int j = 0; j < kMaxSplits / 32; ++j) {
        const float w = M == -INFINITY ? 0.f : ex2(x[j].x - M);
        if (tid < 32) weight[lane + 32 * j] = w;
        sum += w * x[j].y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int b = grp; b < np; b += groups * kCombBatch) {
        if (b > grp) load(b);
#pragma unroll
        for (int j = 0; j < kCombBatch; ++j) {
            if (b + groups * j >= np) break;
            const float w = weight[b + groups * j];
            o4.x = fmaf(w, v[j].x, o4.x);
            o4.y = fmaf(w, v[j].y, o4.y);
            o4.z = fmaf(w, v[j].z, o4.z);
            o4.w = fmaf(w, v[j].w, o4.w);
        }
    }
    if (grp) sh[grp - 1][tid & 63] = o4;
    __syncthreads();
    if (grp) return;
#pragma unroll 1
    for (int j = 0; j < groups - 1; ++j) {
        const float4 y = sh[j][tid];
        o4.x += y.x;
        o4.y += y.y;
        o4.z += y.z;
        o4.w += y.w;
    }
    uint2 pk;
    pk.x = pack_bf16(__fdiv_rn(o4.x, sum), __fdiv_rn(o4.y, sum));
    pk.y = pack_bf16(__fdiv_rn(o4.z, sum), __fdiv_rn(o4.w, sum));
    *reinterpret_cast<uint2 *>(a.out + (int64_t)blockIdx.x * kHeadDim + 4 * (tid & 63)) = pk;
}

// Cost model in nanoseconds, fitted to 124 calls of 2 to 64 streams (128 to 31,000
// shared positions, 100 to 2,000 own, 1 or 4 new tokens, 1 or 2 KV heads of 8
// columns): a coefficient for a pair's tile of 128 shared keys (bf16, e4m3), one for
// its start and end, for a hundred rows of partials written and read again, and for
// the merging kernel.  Within 14 % of each of those calls as the kernel was then.  It
// has become faster since, and a tile's coefficient is above a tile's time: 64
// streams on 31,000 positions 66.6 us modelled, 52.6 measured; 32 of e4m3 pages on
// 24,000 41.4, 34.4; four prompts 32.1, 26.0; eight samples 18.5, 20.0.  Where the
// model is far off, decoding alone costs twice as much and more (60 us for the four
// prompts), so the choice does not hang on it.
constexpr int64_t kTileCost[2] = {2200, 3000}, kPairCost = 7200, kRowsCost = 22, kMergeCost[2] = {4500, 5300};
// ... and of the streams decoded alone: start, a thousand units of the windowed
// plan's cost, a million keys, and what those take more with more than eight columns
// a stream.
constexpr int64_t kAloneCost[2] = {-800, 10000}, kAloneUnits[2] = {2200, 610}, kAloneKeys[2] = {22900, 79600}, kAloneWide[2] = {119000, 178000};

}  // namespace

// Keys are split into whole tiles, each split of any unit up to the same cost `per`,
// so that the pairs fill the GPU about once; the count of splits never passes the
// pairs the GPU holds (or one a unit), which bounds the workspace whatever the
// lengths.  (Units that do not divide the pairs leave some empty: five equal prompts
// at 8 KV heads are 40 splits for 76 pairs.)
void plan_prefix(const Common &c, int nsm, PrefixPlan *plan) {
    const int64_t H = c.n_kv_heads, slots = std::max(1, nsm / 2);
    plan->n_units = 0;
    plan->nsm = nsm;
    int64_t most = 1;  // cost of a unit
    const auto cost_of = [](const PrefixUnit &u) -> int64_t {
        const int64_t tiles = (u.keys + kN - 1) / kN, shared = u.shared / kN;
        return shared * kSharedCost + (tiles - shared) * kOwnCost;
    };
    for (int k = 0; k < plan->n_groups; ++k) {
        PrefixGroup &g = plan->group[k];
        g.unit0 = plan->n_units;
        for (int row0 = 0; row0 < g.rows; row0 += kUnitRows) {
            PrefixUnit &u = plan->unit[plan->n_units++];
            u.layer_base = g.layer_base;
            u.ps = g.ps;
            u.ptok = g.ptok;
            u.n_pages = g.n_pages;
            u.shared = g.shared;
            u.early = g.early;
            u.s0 = g.s0;
            u.n_seqs = g.n_seqs;
            u.tok0 = g.tok0;
            u.map_k = u.map_v = u.map_run = -1;  // (plan_prefix_maps gives it its maps)
            u.layer_row = 0;
            u.row0 = row0;
            u.rows = std::min(kUnitRows, g.rows - row0);
            const auto stream = [&](int row) {
                int s = g.s0;
                for (int t = g.s0; t < g.s0 + g.n_seqs; ++t)
                    if (plan->seq[t].n_new > 0 && plan->seq[t].tok <= g.tok0 + row / c.group) s = t;
                return s;
            };
            u.s_first = stream(row0);
            const PrefixStream &last = plan->seq[stream(row0 + u.rows - 1)];
            const auto pad = [](int n) { return (n + kRun - 1) / kRun * kRun; };
            u.keys = pad(g.shared) + last.own + pad(last.len - g.shared) - plan->seq[u.s_first].own;
            most = std::max(most, cost_of(u));
        }
    }
    const int64_t cap = std::max(H * plan->n_units, slots);
    const int fp8 = c.kv_fp8 ? 1 : 0;
    int64_t chosen = most;
    plan->cost = INT64_MAX;
    for (int64_t k = 1, last = 0; k <= std::min<int64_t>(slots, kMaxSplits); ++k) {
        const int64_t per = std::max<int64_t>(std::max(kSharedCost, kOwnCost), (most + k - 1) / k);
        if (per == last) continue;
        last = per;
        int64_t items = 0, rows = 0;
        for (int i = 0; i < plan->n_units; ++i) {
            const int64_t n = H * ((cost_of(plan->unit[i]) + per - 1) / per);
            items += n;
            rows += n * plan->unit[i].rows;
        }
        if (items > cap) break;  // (more splits have no fewer)
        const int64_t cost = (items + slots - 1) / slots * (per * kTileCost[fp8] / kSharedCost + kPairCost) +
                             (k > 1 ? rows * kRowsCost / 100 + kMergeCost[fp8] : 0);
        if (cost < plan->cost) {
            plan->cost = cost;
            chosen = per;
        }
    }
    int64_t floats = 0;
    plan->items = 0;
    plan->merge = false;
    for (int i = 0; i < plan->n_units; ++i) {
        PrefixUnit &u = plan->unit[i];
        plan->work_off[i] = plan->items;
        u.per = static_cast<int32_t>(std::max<int64_t>(chosen, kOwnCost));
        u.nsplit = static_cast<int32_t>((cost_of(u) + u.per - 1) / u.per);
        u.ws_off = floats;
        plan->items += static_cast<int32_t>(H * u.nsplit);
        if (u.nsplit > 1) {
            plan->merge = true;
            floats += (H * u.nsplit * u.rows * (kHeadDim + 2) + 63) / 64 * 64;
        }
    }
    plan->floats = floats;
}

// Nanoseconds of the streams' windowed decode over all their positions.
int64_t alone_cost(const Common &c, const WindowPlan &plan) {
    const int fp8 = c.kv_fp8 ? 1 : 0;
    bool over8 = false;
    for (int s = 0; s < c.n_seqs; ++s) over8 |= c.seq[s].n_new * c.group > 8;
    return kAloneCost[fp8] + plan.cost * kAloneUnits[fp8] / 1000 +
           plan.keys * (kAloneKeys[fp8] + (over8 ? kAloneWide[fp8] : 0)) / 1000000;
}

// At most `slots` pairs of as many rows as a unit can have (or, with more units
// than that, one split each, which needs none).
size_t prefix_ws_bytes(const Common &c, const pkv_group *groups, int32_t n_groups, int nsm) {
    const int64_t slots = std::max(1, nsm / 2);
    int64_t most = 0;
    int s = 0;
    for (int32_t k = 0; k < n_groups; ++k) {
        int64_t rows = 0;
        for (int32_t i = 0; i < groups[k].n_seqs; ++i) rows += (int64_t)c.seq[s++].n_new * c.group;
        most = std::max(most, std::min<int64_t>(rows, kUnitRows));
    }
    return static_cast<size_t>((slots * most * (kHeadDim + 2) + 64 * kMaxUnits) * 4);
}

int launch_prefix(const Common &c, const PrefixPlan &plan, const DecodeMaps &maps, const uint16_t *q, uint16_t *out, float *ws,
                  cudaStream_t stream) {
    using Kernel = void (*)(DecodeMaps, PrefixArgs);
    const Kernel fns[2][2] = {{prefix_partial<false, false>, prefix_partial<false, true>}, {prefix_partial<true, false>, prefix_partial<true, true>}};
    static std::atomic<uint64_t> attr_done{0};
    if (once_per_device(attr_done, [&] {
            for (int i = 0; i < 4; ++i)
                if (cudaFuncSetAttribute(fns[i >> 1][i & 1], cudaFuncAttributeMaxDynamicSharedMemorySize, i >> 1 ? Lay<true>::smem : Lay<false>::smem) !=
                    cudaSuccess)
                    return PKV_ECUDA;
            return PKV_OK;
        }) != PKV_OK)
        return PKV_ECUDA;
    PrefixArgs a;
    a.q = q;
    a.out = out;
    a.ws = ws;
    a.status = c.status;
    a.n_units = plan.n_units;
    a.n_seqs = plan.n_seqs;
    a.n_kv_heads = c.n_kv_heads;
    a.n_q_heads = c.n_q_heads;
    a.group = c.group;
    std::copy(plan.seq, plan.seq + PKV_MAX_SEQS, a.seq);
    std::copy(plan.unit, plan.unit + plan.n_units, a.unit);
    std::copy(plan.work_off, plan.work_off + plan.n_units, a.work_off);
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
    bool runs = true;
    for (int i = 0; i < plan.n_units; ++i) runs &= plan.unit[i].map_run >= 0;
    if (cudaLaunchKernelEx(&cfg, fns[c.kv_fp8 != 0][runs], maps, a) != cudaSuccess) return PKV_ECUDA;
    if (!plan.merge) return PKV_OK;
    CombineArgs m;
    m.ws = ws;
    m.out = out;
    m.n_groups = plan.n_groups;
    m.n_kv_heads = c.n_kv_heads;
    m.n_q_heads = c.n_q_heads;
    m.group = c.group;
    for (int i = 0; i < plan.n_groups; ++i) {
        m.tok0[i] = plan.group[i].tok0;
        m.unit0[i] = plan.group[i].unit0;
    }
    for (int i = 0; i < plan.n_units; ++i) m.unit[i] = {plan.unit[i].ws_off, plan.unit[i].rows, plan.unit[i].nsplit};
    int64_t tokens = 0;
    for (int s = 0; s < c.n_seqs; ++s) tokens += c.seq[s].n_new;
    const int64_t rows = tokens * c.n_q_heads;
    const int threads = rows <= (int64_t)kCombCtas * plan.nsm ? kCombThreads : kCombThreads / 2;
    return launch_status(launch_pdl(prefix_combine, static_cast<unsigned>(rows), threads, 0, stream, m));
}

}  // namespace pkv
