// Chunk attention over a sliding window with sinks, on the fifth-generation
// tensor cores (tcgen05).
//
// Rows: the (query, head) pairs of one KV head, 128 to an M-tile.  The keys of
// an M-tile are the sinks (padded to whole runs of 16) followed by the
// positions from its first query's window on, counted as virtual keys from 0
// in tiles of 128, so no tile holds keys between the sinks and the window and
// a window of W keys takes about (W + 32) / 128 tiles wherever it lies.
//
// window_gather first copies the rows that the chunk reads (the sinks and the
// first query's window on) out of their pages into the workspace, a KV head's
// rows one after another, K as it is and V in fp16, zeros behind the last
// one: a tile is then one TMA copy whatever the page size, no row that no
// query reads comes near a product, and the PV product runs in fp16 on one P
// part (a bf16 P would need two for the weights' significant bits).  A V
// entry beyond fp16's range makes the output non-finite and is reported.
//
// window_chunk is persistent: a CTA takes every gridDim-th item (an M-tile of
// a split), because a window's items are short (a 1,024-key window is nine
// tiles) and one item's start and end would take as long as its tiles.
//   warps 0-7   softmax: two threads a row, each on 64 of a tile's keys
//   warps 8-11  edge: the next item's Q into tensor memory, this item's O out
//   warp 12     issues the S products, warp 15 the PV products (one thread for
//               both kept the tensor pipe waiting while it waited on barriers
//               and committed: a prompt of 8,192 at a window of 1,024 took 157 us,
//               against 144)
//   warps 13,14 fill a ring of five 16 KB slots each, K and V, by TMA
// Per tile: S = Q K^T -> TMEM, P = softmax numerators in fp16 -> shared memory
// (two buffers: a tile's P is written while the last tile's product runs), O +=
// P V -> TMEM.  Q sits in TMEM (the S product's A operand), and the next item's
// Q goes there, a half at a time, while this item's last tile is in the softmax
// and its PV product; O is read while the next item's first tile is scored.
// O is rescaled only when a row's maximum grows by more than 2^8.
//
// What bounds it: the operands' way through shared memory.  A 128-key tile
// brings 128 KB of K and V in, 32 KB of P are written and the products read
// 160 KB, 2,500 cycles of the memory's width beside 2,600 of the products; a
// tile takes 3,400 (1.75 us).  Beside that the end of an item costs about a tile and a half
// (its masked tiles, its O out, the next item's masked start).  8,192 queries at
// a window of 1,024 (129 GFLOP that some query sees): 136 us, 950 TFLOP/s; 512
// queries at 31,000 with a window of 4,096 (34 GFLOP in 64 items, split over the
// SMs): 53 us, 6 of them the gather and 6 the combine.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kN = 128;              // keys a tile
constexpr int kRun = 16;             // rows of a run (sinks are padded to whole runs)
constexpr int kThreads = 512;
constexpr int kSoftThreads = 256;
constexpr int kEdgeThreads = 128;
constexpr int kWarpS = 12, kWarpV = 14, kWarpPv = 15;  // warp 13 fills the K ring
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kQCol = 0, kSCol = 128, kOCol = 256;
constexpr int kKRegion = kN * 128;   // one 64-dim region of 128 K rows
constexpr int kVKeys = 32;            // keys of a V slot
constexpr int kVRegion = kVKeys * 128;  // one 64-dim region of its rows
constexpr int kSlotBytes = kKRegion; // K of the tile's keys over 64 dims, or V of 32 keys
constexpr int kSlots = 5;            // of each ring
constexpr int kPRegion = kM * 128;   // 64 keys of the 128 P rows
constexpr int kPBuf = 2 * kPRegion;  // P of a tile; two tiles' buffers
constexpr int kOffK = 2 * kPBuf, kOffV = kOffK + kSlots * kSlotBytes;
static_assert(4 * kVRegion == kSlotBytes, "a V slot is 32 keys of four regions");
constexpr int kOffRed = kOffV + kSlots * kSlotBytes;   // [tile parity][half][row] row maxima
constexpr int kOffSum = kOffRed + 2 * 2 * kM * 4;         // [row] sums of an item
constexpr int kOffBar = kOffSum + kM * 4;
enum Bars {
    kKFull = 0,            // a ring's slots: filled, and free again
    kKEmpty = kSlots,
    kVFull = 2 * kSlots,
    kVEmpty = 3 * kSlots,
    kSFull = 4 * kSlots,  // S of a tile is in TMEM
    kSEmpty,              // ... and has been read
    kPFull,               // P of an even or odd tile is in shared memory (two barriers)
    kODone = kPFull + 2,  // an even or odd tile's PV product is done (two barriers)
    kQFull = kODone + 2,               // a half of an item's Q is in TMEM (two barriers)
    kQEmpty = kQFull + 2, // ... and its last S product is done
    kOLast,               // an item's last PV product is done
    kOFree,               // ... and its O and sums have been read
    kSums,                // an item's sums are in shared memory
    kRed,                 // a tile's half-row maxima are in shared memory
    kDrain,               // a failed issuer's products are done (S, PV)
    kNumBars = kDrain + 2
};
constexpr int kSmem = kOffBar + kNumBars * 8 + 16;
static_assert(kSmem <= 232448, "above the 227 KB a CTA may hold");
constexpr float kScaleLog2 = 0.0625f * 1.4426950408889634f;  // log2(e) / sqrt(256)
constexpr float kRescale = 8.f;  // rescale O when the max grows by more than 2^8
// Row maxima beyond this (log2 units) are reported: float32 steps of 4 and more
// lie between scores there, and the reference's own rounding, up to half a step,
// would take P out of fp16's range.
constexpr float kFarScore = 67108864.f;  // 2^26

struct ChunkArgs {
    const uint16_t *q;
    uint16_t *out;
    float *ws;
    uint16_t *rows16;   // the gathered rows: K, then V in fp16
    int64_t n_rows;     // rows of each
    int32_t window, n_sink, n_items;
    int32_t split;      // whether some stream's M-tiles are split
    int32_t map_k, map_v, map_run;
    int32_t row0[PKV_MAX_SEQS];  // first gathered row of the stream (KV head 0)
};

// The gathered rows of one KV head of a stream: positions below `sinks` at
// their own index, positions from lo on from row `win` on, zero rows between
// and behind (`rows` counts up to the last position's).  The sinks are padded
// to whole runs; where that reaches the window's start, win == lo and every
// row's index is its position.
struct Gathered {
    int32_t lo, sinks, win, rows, stride;
};
__host__ __device__ inline Gathered gathered(int32_t len, int32_t n_new, int32_t window, int32_t n_sink) {
    Gathered g;
    g.lo = len - n_new + 1 - window;
    if (g.lo < 0) g.lo = 0;
    g.sinks = n_sink < g.lo ? n_sink : g.lo;
    g.win = (g.sinks + kRun - 1) / kRun * kRun;
    if (g.win > g.lo) g.win = g.lo;
    g.rows = g.win + (len - g.lo);
    g.stride = (g.rows + kRun - 1) / kRun * kRun + kN;  // a last tile reads up to kN - 1 rows more
    return g;
}

// The virtual keys of an M-tile whose queries sit at positions qf .. ql: the
// sinks' runs (sink_end keys, the positions below slim of them read), then
// the positions from lo on.
struct Keys {
    int32_t lo, slim, sink_end, total;
};
__host__ __device__ inline Keys keys_of(const Gathered &g, int32_t qf, int32_t ql, int32_t window, int32_t n_sink) {
    Keys k;
    k.lo = qf + 1 - window;
    if (k.lo < 0) k.lo = 0;
    // where rows are positions, sinks that (nearly) reach the window and it are
    // one run from position 0 on
    if (g.win == g.lo && k.lo - kRun <= n_sink) k.lo = 0;
    k.slim = k.lo > 0 ? n_sink : 0;
    k.sink_end = (k.slim + kRun - 1) / kRun * kRun;
    k.total = k.sink_end + (ql - k.lo + 1);
    return k;
}

struct Item {
    Keys k;
    int s, kvh, split, col0, rows, key0, ntiles;
};

__device__ __forceinline__ Item item_at(const Common &c, const ChunkArgs &a, int i) {
    Item t;
    t.s = find_seq(c.n_seqs, i, [&](int j) { return c.seq[j].work_off; });
    const SeqDev &sd = c.seq[t.s];
    const int mtiles = (sd.ncols + kM - 1) / kM;
    const int r = i - sd.work_off, u = r / mtiles;
    t.col0 = (r - u * mtiles) * kM;
    t.kvh = u / sd.nsplit;
    t.split = u - t.kvh * sd.nsplit;
    t.rows = min(kM, sd.ncols - t.col0);
    const int qbase = sd.len - sd.n_new;
    const Gathered g = gathered(sd.len, sd.n_new, a.window, a.n_sink);
    t.k = keys_of(g, qbase + t.col0 / c.group, qbase + (t.col0 + t.rows - 1) / c.group, a.window, a.n_sink);
    t.key0 = t.split * sd.split_len;
    const int key1 = min(t.k.total, t.key0 + sd.split_len);
    // a split past a short M-tile's keys scores one tile, all of it masked
    t.ntiles = max(1, (key1 - t.key0 + kN - 1) / kN);
    return t;
}

// V slots of the tile of virtual keys v0 .. (keys past `total` have no weight;
// a tile past it, all masked, takes one).
__device__ __forceinline__ int v_slots(int v0, int total) {
    return max(1, min(kN / kVKeys, (total - v0 + kVKeys - 1) / kVKeys));
}

// Gathered row of virtual key v of an item.
__device__ __forceinline__ int row_of(const Gathered &g, const Keys &k, int v) {
    if (v < k.sink_end || g.win == g.lo) return v < k.sink_end ? v : k.lo + (v - k.sink_end);
    return g.win + (k.lo - g.lo) + (v - k.sink_end);
}

// The lowest n of 64 bits.
__device__ __forceinline__ uint64_t below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Two float32 operations an instruction, each rounded as alone: the softmax and
// edge warps' issue slots count (a prompt of 8,192 took 141.0 us with single
// ones, 135.9 with these).
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}

// Transpose over each four lanes: word j of lane i goes to word i of lane j.
// Rows that lie one a lane are so read and written 64 bytes of a row at a time
// by four lanes (16 bytes of 32 rows an instruction, as the lanes hold them,
// kept the load and store units of an item's Q and O busy for 8,000 cycles).
__device__ __forceinline__ uint4 shfl_xor16(const uint4 &v, int m) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                      __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m));
}
__device__ __forceinline__ uint4 pick(bool b, const uint4 &x, const uint4 &y) {
    return make_uint4(b ? x.x : y.x, b ? x.y : y.y, b ? x.z : y.z, b ? x.w : y.w);
}
__device__ __forceinline__ void quad_transpose(uint4 *v, int lane) {
    const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
    for (int p = 0; p < 4; p += 2) {
        const uint4 got = shfl_xor16(pick(b0, v[p], v[p + 1]), 1);
        v[p] = pick(b0, got, v[p]);
        v[p + 1] = pick(b0, v[p + 1], got);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint4 got = shfl_xor16(pick(b1, v[p], v[p + 2]), 2);
        v[p] = pick(b1, got, v[p]);
        v[p + 2] = pick(b1, v[p + 2], got);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    window_chunk(const __grid_constant__ Common c, const __grid_constant__ DecodeMaps maps,
                 const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    {
        // the address as the hardware gives it (an asm result the compiler
        // cannot fold from the declared alignment)
        uint32_t base;
        asm volatile("mov.u32 %0, %1;" : "=r"(base) : "r"(smem_u32(smem)));
        if (base & 1023u) {  // uniform: every thread returns before any barrier
            if (tid == 0 && c.status) atomicOr(c.status, PKV_DEV_SMEM);
            return;
        }
    }
    const int H = c.n_kv_heads, G = c.group;
    if (tid == 0) {
        for (int i = 0; i < kSFull; ++i) mbar_init(&bars[i], 1);  // both rings
        mbar_init(&bars[kSFull], 1);
        mbar_init(&bars[kSEmpty], kSoftThreads);
        mbar_init(&bars[kPFull], kSoftThreads);
        mbar_init(&bars[kPFull + 1], kSoftThreads);
        mbar_init(&bars[kODone], 1);
        mbar_init(&bars[kODone + 1], 1);
        mbar_init(&bars[kQFull], kEdgeThreads);
        mbar_init(&bars[kQFull + 1], kEdgeThreads);
        mbar_init(&bars[kQEmpty], 1);
        mbar_init(&bars[kOLast], 1);
        mbar_init(&bars[kOFree], kEdgeThreads);
        mbar_init(&bars[kSums], kSoftThreads);
        mbar_init(&bars[kRed], kSoftThreads);
        mbar_init(&bars[kDrain], 1);
        mbar_init(&bars[kDrain + 1], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < kM) reinterpret_cast<float *>(smem + kOffSum)[tid] = 0.f;
    // tcgen05 alloc, dealloc, ld and st are warp-collective (.sync.aligned):
    // every one follows a __syncwarp, because a CTA barrier does not
    // reconverge a warp whose lanes took different paths before it
    if (warp == kWarpS) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = smem_u32(smem);
    if (tid == 0) pdl_trigger();  // this grid writes nothing that is read before a grid-dependency wait

    // Every wait is bounded; a role whose wait runs out raises the flag and
    // leaves its loops, and so do, a second later, the roles that wait for it.
    auto wait = [&](int bar, uint32_t phase) -> bool {
        const bool ok = mbar_wait(&bars[bar], phase & 1, c.status);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    auto wait_warp = [&](int bar, uint32_t phase) -> bool {
        return __all_sync(0xffffffffu, wait(bar, phase));
    };

    int last_q = -1;  // a producer's last slot
    if (warp < 8) {
        // ------- softmax: row r (TMEM lane r) by two threads, keys 64 hf .. 64 hf + 63 of a tile -------
        const int r = lane + 32 * (warp & 3), hf = warp >> 2;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float *const red = reinterpret_cast<float *>(smem + kOffRed);
        uint8_t *const p_row = smem + hf * kPRegion + r * 128;
        // positions fit 31 bits, sums of two of them clamped to 30 do
        constexpr int kFar = 1 << 30;
        const int n_sink = min(a.n_sink, kFar);
        uint32_t T = 0, it = 0;  // tiles and items so far
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.n_items; i += gridDim.x, ++it) {
            const Item t = item_at(c, a, i);
            const SeqDev &sd = c.seq[t.s];
            // rows past the M-tile's end take no mask: their Q rows are
            // zero, so their scores are finite, and they are never written
            const int qpos = r < t.rows ? sd.len - sd.n_new + (t.col0 + r) / G : kFar;
            const int win0 = r < t.rows ? max(qpos - a.window, -kFar) : -kFar;  // keys above it are in the row's window
            float m_used = -INFINITY, l = 0.f;
            for (int n = 0; n < t.ntiles; ++n, ++T) {
                if (!(ok = wait_warp(kSFull, T))) break;
                tc_fence_after();
                uint32_t sv[64];
                tmem_ld64(lane_base + kSCol + 64 * hf, sv);
                tc_fence_before();
                mbar_arrive(&bars[kSEmpty]);
                const int v0 = t.key0 + n * kN + 64 * hf;             // this thread's first virtual key
                const int kp0 = v0 - t.k.sink_end + t.k.lo;            // its position, in the window's part
                float x[64];
#pragma unroll
                for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(sv[j]);
                const bool all = v0 >= t.k.sink_end
                                     ? kp0 + 63 <= qpos && (kp0 > win0 || kp0 + 63 < n_sink)
                                     : v0 + 63 < t.k.slim;
                if (!__all_sync(0xffffffffu, all)) {
                    // one bit a key: the sinks' runs hold positions below slim,
                    // the window's part positions up to qpos that are in the
                    // row's window or among the sinks.  Compared key by key this
                    // took 3 to 4 us a tile, a fifth of a nine-tile item.  (Leaving
                    // 16 keys alone that every row sees cost the other tiles more
                    // than it saved these.)
                    const uint64_t part = below(t.k.sink_end - v0);
                    const uint64_t see = (part & below(t.k.slim - v0)) |
                                         (~part & below(qpos - kp0 + 1) & (~below(win0 - kp0 + 1) | below(n_sink - kp0)));
                    const uint32_t lo = static_cast<uint32_t>(see), hi = static_cast<uint32_t>(see >> 32);
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (!((j < 32 ? lo : hi) & (1u << (j & 31)))) x[j] = -INFINITY;
                }
                // this half's max as eight interleaved chains, then the row's
                // from the partner thread, in float32 (a reference above the
                // maximum, by a coarser rounding of large scores, takes P out of
                // fp16's range)
                float m8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) m8[j] = x[j];
#pragma unroll
                for (int j = 8; j < 64; ++j) m8[j & 7] = fmaxf(m8[j & 7], x[j]);
                const float lmx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                        fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                red[((T & 1) * 2 + hf) * kM + r] = lmx;
                mbar_arrive(&bars[kRed]);
                if (!(ok = wait_warp(kRed, T))) break;
                const float mx = fmaxf(lmx, red[((T & 1) * 2 + (hf ^ 1)) * kM + r]) * kScaleLog2;  // log2 units; -inf when the whole row of the tile is masked
                const bool grow = m_used != -INFINITY && mx > m_used + kRescale;
                if (__any_sync(0xffffffffu, grow)) {
                    // correct this thread's half of O: the previous tile's
                    // products must be in it first (some row of the warp had a
                    // maximum before, so this is not the item's first tile)
                    if (!(ok = wait_warp(kODone + ((T - 1) & 1), (T - 1) >> 1))) break;
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
                    m_used = mx;  // nothing accumulated yet: O is still zero
                }
                // p = 2^(s * scale - m); a masked score is -inf and gives 0 (the
                // offset is 0 while every score so far was masked).  fp16: 11
                // significant bits, weights at most 2^8 with the lazy rescale
                const float m_off = m_used == -INFINITY ? 0.f : m_used;
                const float2 scale = make_float2(kScaleLog2, kScaleLog2), off = make_float2(-m_off, -m_off);
                float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t p16[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float2 p = fma2(make_float2(x[j], x[j + 1]), scale, off);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    ps[(j >> 1) & 1] = add2(ps[(j >> 1) & 1], p);
                    p16[j / 2] = pack_f16(p.x, p.y);
                }
                l += (ps[0].x + ps[1].x) + (ps[0].y + ps[1].y);
                // this buffer's P rows are free once the products of the tile
                // before the last are done
                if (T > 1 && !(ok = wait_warp(kODone + (T & 1), (T >> 1) - 1))) break;
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                    *reinterpret_cast<uint4 *>(p_row + (T & 1) * kPBuf + ((ch ^ (r & 7)) << 4)) =
                        make_uint4(p16[4 * ch], p16[4 * ch + 1], p16[4 * ch + 2], p16[4 * ch + 3]);
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&bars[kPFull + (T & 1)]);
            }
            if (!ok) break;
            // the row's sum, for the edge warps, from zero (two terms: the same in
            // either order)
            if (it > 0 && !(ok = wait_warp(kOFree, it - 1))) break;
            atomicAdd(reinterpret_cast<float *>(smem + kOffSum) + r, l);
            mbar_arrive(&bars[kSums]);
            if (hf == 0) {
                // (rows past the M-tile's end score 0)
                if (m_used != -INFINITY && fabsf(m_used) > kFarScore && c.status) atomicOr(c.status, PKV_DEV_RANGE);
                if (a.split) {
                    // a split's maximum, to the workspace (the scores came of tiles
                    // copied behind the grid-dependency wait: the last call is done
                    // with it); a finite one for NaN and infinity, whose sums the
                    // combine takes as they are.  The item is looked up anew: kept along the tiles it
                    // would not fit the registers
                    int again = i;
                    asm volatile("" : "+r"(again));
                    const Item e = item_at(c, a, again);
                    const SeqDev &se = c.seq[e.s];
                    float *const part_ml = a.ws + se.ws_off + (int64_t)H * se.nsplit * se.ncols * kHeadDim;
                    if (se.nsplit > 1 && r < e.rows)
                        part_ml[2 * (((int64_t)e.kvh * se.nsplit + e.split) * se.ncols + e.col0 + r)] = fminf(m_used, FLT_MAX);
                }
            }
        }
    } else if (warp < kWarpS) {
        // ------- edge: Q into TMEM columns 0-127 (bf16 pairs), O out -------
        pdl_wait();
        const int r = lane + 32 * (warp & 3);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        auto q_row = [&](const Item &t) -> int64_t {  // packed row of this thread's query row
            const int col = t.col0 + r, j = col / G;
            return ((int64_t)c.seq[t.s].tok_off + j) * c.n_q_heads + t.kvh * G + (col - j * G);
        };
        // A half of the rows' Q (128 dims) from global memory, and into TMEM
        const int quad = lane & ~3, word = lane & 3;
        uint4 qv[16];
        auto load_q = [&](const Item &t, int half) {
            const int64_t mine = r < t.rows ? q_row(t) : -1;
            int64_t row[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) row[i] = shfl64(mine, quad + i);
#pragma unroll
            for (int j = 0; j < 16; j += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qv[j + i] = row[i] >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.q + row[i] * kHeadDim + 128 * half) + j + word)
                                            : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 16; j += 4) quad_transpose(qv + j, lane);
        };
        auto put_q = [&](int half) {
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    w[4 * j] = qv[8 * ch + j].x;
                    w[4 * j + 1] = qv[8 * ch + j].y;
                    w[4 * j + 2] = qv[8 * ch + j].z;
                    w[4 * j + 3] = qv[8 * ch + j].w;
                }
                __syncwarp();
                tmem_st32(lane_base + kQCol + 64 * half + 32 * ch, w);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            mbar_arrive(&bars[kQFull + half]);
        };
        uint32_t it = 0;
        Item t = item_at(c, a, blockIdx.x);
        load_q(t, 0);
        put_q(0);
        load_q(t, 1);
        put_q(1);
        for (int i = blockIdx.x; i < a.n_items; i += gridDim.x, ++it) {
            const int next = i + gridDim.x;
            Item t2 = t;
            if (next < a.n_items) {
                // the first half waits in registers for the last product that
                // reads this item's Q, the second in L2
                t2 = item_at(c, a, next);
                load_q(t2, 0);
                if (r < t2.rows)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + q_row(t2) * kHeadDim + 128 + 64 * j));
                if (!wait_warp(kQEmpty, it)) break;
                tc_fence_after();
                put_q(0);
                load_q(t2, 1);
                put_q(1);
            }
            if (!wait_warp(kSums, it)) break;
            if (!wait_warp(kOLast, it)) break;
            tc_fence_after();
            const SeqDev &sd = c.seq[t.s];
            const bool row_ok = r < t.rows, single = sd.nsplit == 1;
            float *const sum = reinterpret_cast<float *>(smem + kOffSum) + r;
            const float l = *sum;
            *sum = 0.f;
            const float inv = 1.f / l;  // (0 only where every score is -infinity: NaN)
            const int64_t prow = ((int64_t)t.kvh * sd.nsplit + t.split) * sd.ncols + t.col0 + r;
            const int64_t mine = !row_ok ? -1 : single ? q_row(t) : prow;  // output row, or the partials'
            int64_t row[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) row[j] = shfl64(mine, quad + j);
            float *part_acc = a.ws + sd.ws_off;
            float *part_ml = part_acc + (int64_t)H * sd.nsplit * sd.ncols * kHeadDim;
            float2 odd = make_float2(0.f, 0.f);  // NaN once a sum is not finite: a V entry beyond fp16's range
#pragma unroll 1
            for (int ch = 0; ch < 8; ++ch) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(lane_base + kOCol + 32 * ch, o);
                if (ch == 7) {  // the next item's first PV product may write O
                    tc_fence_before();
                    mbar_arrive(&bars[kOFree]);
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    odd = fma2(make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), make_float2(0.f, 0.f), odd);
                if (single) {
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = 8 * j + 2 * e;
                            const float2 z = mul2(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), make_float2(inv, inv));
                            w[e] = pack_bf16(z.x, z.y);
                        }
                        v[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    quad_transpose(v, lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (row[j] >= 0) *(reinterpret_cast<uint4 *>(a.out + row[j] * kHeadDim + 32 * ch) + word) = v[j];
                } else {
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
                                *(reinterpret_cast<uint4 *>(part_acc + row[j] * kHeadDim + 32 * ch + 16 * h) + word) = v[j];
                    }
                }
            }
            // (its maximum: the softmax warps.  A sum that is NaN comes with an O
            // that is, which the combine divides only by a sum above zero)
            if (row_ok && !single) part_ml[prow * 2 + 1] = l == l ? l : 1.f;
            if (row_ok && (odd.x + odd.y != 0.f || (single && !(l > 0.f))) && c.status) atomicOr(c.status, PKV_DEV_RANGE);
            t = t2;
        }
    } else if (warp == kWarpS || warp == kWarpPv) {
        if (lane == 0) {
            // ---------------- MMA issue ----------------
            // operands written by threads (Q, P) were fenced by their writers
            // before they arrived.  A descriptor's address is its low 14 bits in
            // units of 16 bytes, and shared memory ends below 256 KB: offsets
            // are added to it.
            uint32_t q = 0, T = 0, it = 0;  // slots, tiles and items so far
            bool ok = true;
            auto take = [&](int full, int ring, uint32_t &addr) -> bool {
                if (!wait(full + q % kSlots, q / kSlots)) return false;
                tc_fence_after();
                addr = sbase + ring + (q % kSlots) * kSlotBytes;
                return true;
            };
            auto give = [&](int empty) {
                tc_commit(&bars[empty + q % kSlots]);  // free once these MMAs are done
                ++q;
            };
            if (warp == kWarpS) {
                const uint32_t idesc = mma_idesc(kN, false);
                const uint64_t desc_k = smem_desc(0, 16, 1024);
                int ntiles = item_at(c, a, blockIdx.x).ntiles, next_tiles = 0;
                for (int i = blockIdx.x; ok && i < a.n_items; i += gridDim.x, ++it, ntiles = next_tiles) {
                    for (int n = 0; ok && n < ntiles; ++n, ++T) {
                        if (T > 0 && !(ok = wait(kSEmpty, T - 1))) break;
                        tc_fence_after();
                        // S = Q K^T, 64 dims a slot
#pragma unroll 1
                        for (int qt = 0; qt < 4; ++qt) {
                            if (n == 0 && qt % 2 == 0 && !(ok = wait(kQFull + qt / 2, it))) break;
                            uint32_t kb;
                            if (!(ok = take(kKFull, kOffK, kb))) break;
                            const uint64_t dk = desc_k + (kb >> 4);
#pragma unroll
                            for (int k4 = 0; k4 < 4; ++k4)
                                tc_mma_ts(tmem + kSCol, tmem + kQCol + (4 * qt + k4) * 8, dk + (k4 * 32 >> 4), idesc,
                                          (qt > 0 || k4 > 0) ? 1u : 0u);
                            give(kKEmpty);
                        }
                        if (!ok) break;
                        tc_commit(&bars[kSFull]);
                        if (n + 1 == ntiles) tc_commit(&bars[kQEmpty]);
                        // looked up here, while the first product runs
                        if (n == 0 && i + (int)gridDim.x < a.n_items) next_tiles = item_at(c, a, i + gridDim.x).ntiles;
                    }
                }
            } else {
                const uint32_t idesc = mma_idesc(kHeadDim, true, true);
                const uint64_t desc_v = smem_desc(0, kVRegion, 1024), desc_p = smem_desc(sbase, 16, 1024);
                Item t = item_at(c, a, blockIdx.x);
                for (int i = blockIdx.x; ok && i < a.n_items; i += gridDim.x, ++it) {
                    const int ntiles = t.ntiles, key0 = t.key0, total = t.k.total;
                    for (int n = 0; ok && n < ntiles; ++n, ++T) {
                        const int nv = v_slots(key0 + n * kN, total);
                        if (!(ok = wait(kPFull + (T & 1), T >> 1))) break;
                        if (n == 0 && it > 0 && !(ok = wait(kOFree, it - 1))) break;
                        tc_fence_after();
                        // O += P V, 32 keys a slot
#pragma unroll 1
                        for (int vs = 0; vs < nv; ++vs) {
                            uint32_t vb;
                            if (!(ok = take(kVFull, kOffV, vb))) break;
                            const uint64_t dp = desc_p + (((T & 1) * kPBuf + (vs >> 1) * kPRegion + (vs & 1) * 64) >> 4), dv = desc_v + (vb >> 4);
#pragma unroll
                            for (int k2 = 0; k2 < 2; ++k2)
                                tc_mma(tmem + kOCol, dp + (k2 * 32 >> 4), dv + (k2 * 2048 >> 4), idesc,
                                       (n > 0 || vs > 0 || k2 > 0) ? 1u : 0u);
                            give(kVEmpty);
                        }
                        if (!ok) break;
                        tc_commit(&bars[kODone + (T & 1)]);
                        if (n + 1 == ntiles) tc_commit(&bars[kOLast]);
                        if (n == 0 && i + (int)gridDim.x < a.n_items) t = item_at(c, a, i + gridDim.x);
                    }
                }
            }
            if (!ok) {  // no product is in flight when the tensor memory goes
                const int drain = kDrain + (warp == kWarpPv);
                tc_commit(&bars[drain]);
                mbar_wait(&bars[drain], 0, nullptr);
            }
        }
    } else {
        // ------- producers of K slots (64 dims each) and V slots (32 keys each) -------
        pdl_wait();
        const bool is_v = warp == kWarpV;
        const uint64_t pol = policy_evict_normal();  // neighbouring M-tiles read the same rows
        const void *const map = &maps.map[is_v ? a.map_v : a.map_k];
        const void *const map_run = &maps.map[a.map_run];
        const int full0 = is_v ? kVFull : kKFull, empty0 = is_v ? kVEmpty : kKEmpty, ring = is_v ? kOffV : kOffK;
        uint32_t q = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < a.n_items; i += gridDim.x) {
            const Item t = item_at(c, a, i);
            const SeqDev &sd = c.seq[t.s];
            const Gathered g = gathered(sd.len, sd.n_new, a.window, a.n_sink);
            const int base = a.row0[t.s] + t.kvh * g.stride + (is_v ? static_cast<int>(a.n_rows) : 0);
            for (int m = 0; ok && m < t.ntiles; ++m) {
                // (a split past the item's keys copies the first ones, all masked)
                const int v0 = (t.key0 < t.k.total ? t.key0 : 0) + m * kN;
                const bool mixed = v0 < t.k.sink_end && v0 + kN > t.k.sink_end;
                const int n_slots = is_v ? v_slots(t.key0 + m * kN, t.k.total) : 4;
                for (int j = 0; j < n_slots; ++j, ++q) {
                    const uint32_t slot = q % kSlots;
                    if (q >= kSlots && !(ok = wait_warp(empty0 + slot, q / kSlots - 1))) break;
                    uint64_t *const full = &bars[full0 + slot];
                    uint8_t *const dst = smem + ring + slot * kSlotBytes;
                    if (lane == 0) mbar_arrive_expect_tx(full, kSlotBytes);
                    __syncwarp();
                    if (!mixed) {
                        if (lane == 0) {
                            if (is_v) tma_load_3d(dst, map, 0, base + row_of(g, t.k, v0 + kVKeys * j), 0, full, pol);
                            else tma_load_3d(dst, map, 0, base + row_of(g, t.k, v0), j, full, pol);
                        }
                    } else if (lane < 8) {
                        // the sinks' last tile: 16-row runs, one 64-dim box a lane
                        if (is_v) {
                            const int rn = lane >> 2, ch = lane & 3;
                            tma_load_2d(dst + ch * kVRegion + rn * 2048, map_run, 64 * ch,
                                        base + row_of(g, t.k, v0 + kVKeys * j + 16 * rn), full, pol);
                        } else {
                            tma_load_2d(dst + lane * 2048, map_run, 64 * j, base + row_of(g, t.k, v0 + 16 * lane), full, pol);
                        }
                    }
                    __syncwarp();
                    last_q = static_cast<int>(q);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // after a wait that ran out, the copies issued land before the memory goes
    // (this producer's last slots; no later phase has been armed)
    if (*abort_flag)
        for (int k = last_q; k >= 0 && k > last_q - kSlots; --k)
            mbar_wait(&bars[(warp == kWarpV ? kVFull : kKFull) + k % kSlots], (k / kSlots) & 1, nullptr);
    if (warp == kWarpS) {
        __syncwarp();  // lane 0 issued the MMAs, lanes 1-31 went straight here
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The rows a chunk reads, out of their pages: a warp a run of 16 rows of K or
// of V (fp16) of one KV head, a lane 16 bytes of each row, all 16 loads issued
// before any store.  Lane i looks row i up.  A table entry outside
// [0, n_pages) is reported and read as page 0.
constexpr int kGatherThreads = 128;
constexpr int kGatherWarps = kGatherThreads / 32;

__global__ void __launch_bounds__(kGatherThreads)
    window_gather(const __grid_constant__ Common c, const __grid_constant__ ChunkArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t run = (int64_t)blockIdx.x * kGatherWarps + (threadIdx.x >> 5);
    pdl_trigger();  // the chunk kernel waits for this grid before it reads the rows
    const int64_t runs = a.n_rows / kRun;
    if (run >= 2 * runs) return;
    const bool is_v = run >= runs;
    const int row0 = static_cast<int>(is_v ? run - runs : run) * kRun;
    int s = 0;
    for (int t = 0; t < c.n_seqs; ++t)
        if (a.row0[t] >= 0 && row0 >= a.row0[t]) s = t;
    const SeqDev &sd = c.seq[s];
    const Gathered g = gathered(sd.len, sd.n_new, a.window, a.n_sink);
    const int local = row0 - a.row0[s], kvh = local / g.stride;
    // position of row i of the run (-1: a zero row)
    const int i = local - kvh * g.stride + (lane & (kRun - 1));
    const int pos = i < g.sinks ? i : (i >= g.win && i < g.rows) ? g.lo + (i - g.win) : -1;
    const uint16_t *src = nullptr;
    if (pos >= 0) {
        uint32_t *st = lane < kRun && !is_v ? c.status : nullptr;
        src = is_v ? v_row(sd, c.n_kv_heads, kvh, pos, st) : k_row(sd, c.n_kv_heads, kvh, pos, st);
    }
    pdl_wait();  // the chunk's rows were stored by an earlier kernel
    uint4 v[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(shfl64(reinterpret_cast<int64_t>(src), k));
        v[k] = make_uint4(0, 0, 0, 0);
        if (p)  // volatile: the loads stay ahead of the stores
            asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                         : "l"(p + 8 * lane));
    }
    uint16_t *dst = a.rows16 + ((is_v ? a.n_rows : 0) + row0) * kHeadDim + 8 * lane;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
        uint4 w = v[k];
        if (is_v) {  // bf16 -> fp16: exact for 2^-14 to 65,280, 2^-24 steps below
            uint32_t *e = &w.x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                e[j] = pack_f16(__uint_as_float(e[j] << 16), __uint_as_float(e[j] & 0xffff0000u));
        }
        *reinterpret_cast<uint4 *>(dst + (int64_t)k * kHeadDim) = w;
    }
}

// Split model of plan_window_prefill, in hundredths of a microsecond.
constexpr int64_t kTileCost = 175;    // a 128-key tile of one M-tile
constexpr int64_t kItemCost = 300;    // an item's fixed cost
constexpr int64_t kStartCost = 1000;  // a call's first item and the combine of a split call
constexpr int kMaxSplits = 32;

}  // namespace

int plan_window_prefill(Common &c, int32_t window, int32_t n_sink, int nsm, DecodePlan *plan) {
    int64_t items = 0, rows = 0, floats = 0, comb = 0;
    const int H = c.n_kv_heads;
    for (int s = 0; s < c.n_seqs; ++s) {
        SeqDev &d = c.seq[s];
        d.work_off = static_cast<int32_t>(items);
        d.comb_off = static_cast<int32_t>(comb);
        d.ws_off = floats;
        d.ncols = d.n_new * c.group;
        d.nsplit = 1;
        d.split_len = kN;
        if (d.ncols == 0) continue;
        const int mtiles = (d.ncols + kM - 1) / kM;
        // at most: a window, the queries of an M-tile, the sinks' runs
        const int64_t span = std::min<int64_t>(d.n_new, kM / c.group + 2);
        const int64_t most = std::min<int64_t>((int64_t)d.len + kRun, (int64_t)window + n_sink + span + 2 * kRun);
        const int tiles = static_cast<int>((most + kN - 1) / kN);
        // Splits: the count with the least modelled time for this stream alone
        // on nsm SMs (its bits must not depend on its batch).
        const int64_t units = (int64_t)H * mtiles;
        int64_t best = INT64_MAX;
        for (int n = 1; n <= std::min(kMaxSplits, tiles); ++n) {
            const int64_t waves = (units * n + nsm - 1) / nsm;
            const int64_t cost = waves * (((tiles + n - 1) / n) * kTileCost + kItemCost) + (n > 1 ? kStartCost : 0);
            if (cost < best) {
                best = cost;
                d.nsplit = n;
            }
        }
        const int per = (tiles + d.nsplit - 1) / d.nsplit;
        d.split_len = per * kN;
        d.nsplit = (tiles + per - 1) / per;
        items += units * d.nsplit;
        rows += (int64_t)H * gathered(d.len, d.n_new, window, n_sink).stride;
        if (d.nsplit > 1) {
            comb += (int64_t)H * d.ncols * comb_ctas(d.nsplit);
            floats += (int64_t)H * d.nsplit * d.ncols * (kHeadDim + 2);
            floats = (floats + 63) / 64 * 64;
        }
    }
    if (items > INT32_MAX / 2 || comb > INT32_MAX || rows > (1 << 29)) return PKV_EINVAL;
    plan->total_items = static_cast<int32_t>(items);
    plan->total_comb = static_cast<int32_t>(comb);
    plan->ws_bytes = static_cast<size_t>(floats) * 4 + static_cast<size_t>(rows) * 2 * kHeadDim * 2;
    return PKV_OK;
}

int launch_window_prefill(const Common &c, const DecodePlan &plan, int32_t window, int32_t n_sink,
                          const uint16_t *q, uint16_t *out, float *ws, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    if (once_per_device(attr_done, [] {
            return cuda_rc(cudaFuncSetAttribute(window_chunk, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
        }) != PKV_OK)
        return PKV_ECUDA;
    int nsm = 0;
    if (sm_count(&nsm) != PKV_OK) return PKV_ECUDA;
    ChunkArgs a;
    a.q = q;
    a.out = out;
    a.ws = ws;
    a.window = window;
    a.n_sink = n_sink;
    a.n_items = plan.total_items;
    a.split = plan.total_comb > 0;
    int64_t rows = 0;
    for (int s = 0; s < PKV_MAX_SEQS; ++s) {
        a.row0[s] = -1;
        if (s >= c.n_seqs || c.seq[s].ncols == 0) continue;
        a.row0[s] = static_cast<int32_t>(rows);
        rows += (int64_t)c.n_kv_heads * gathered(c.seq[s].len, c.seq[s].n_new, window, n_sink).stride;
    }
    a.n_rows = rows;
    // the gathered rows lie behind the split partials
    a.rows16 = reinterpret_cast<uint16_t *>(reinterpret_cast<char *>(ws) + plan.ws_bytes - (size_t)rows * 2 * kHeadDim * 2);
    // one view of K and V rows: boxes of a K slot, of a V slot and of 16 rows
    // (the maps' type is bf16; a copy moves fp16 rows' bits unchanged)
    DecodeMaps maps;
    int n_maps = 0;
    a.map_k = row_map(maps, n_maps, a.rows16, static_cast<uint64_t>(2 * rows), false, true, kN, 1);
    a.map_v = row_map(maps, n_maps, a.rows16, static_cast<uint64_t>(2 * rows), false, true, kVKeys, 4);
    a.map_run = row_map(maps, n_maps, a.rows16, static_cast<uint64_t>(2 * rows), false);
    if (a.map_k < 0 || a.map_v < 0 || a.map_run < 0) return PKV_ECUDA;
    const int64_t warps = 2 * rows / kRun;
    if (launch_pdl(window_gather, static_cast<unsigned>((warps + kGatherWarps - 1) / kGatherWarps), kGatherThreads, 0,
                   stream, c, a) != cudaSuccess)
        return PKV_ECUDA;
    if (launch_pdl(window_chunk, static_cast<unsigned>(std::min(plan.total_items, nsm)), kThreads, kSmem, stream, c,
                   maps, a) != cudaSuccess)
        return PKV_ECUDA;
    if (plan.total_comb > 0) return launch_combine(c, plan, q, out, ws, stream);
    return PKV_OK;
}

}  // namespace pkv
