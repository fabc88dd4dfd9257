// Decode attention over a sliding window with sinks: a query at position p
// reads the keys j <= p with j > p - window or j < n_sink.
//
// The keys that some query of a stream reads are its first n_sink positions
// and a run that ends at its newest one.  They are counted through as virtual
// keys (WindowSpan): the sinks' 16-key tiles, then the window's, so the rows
// between them are never touched and their pages may be gone.  A tile's keys
// that no query of the stream sees take the row of a neighbouring key that
// one sees, so that nothing stale (a NaN, a page that is gone) reaches an MMA.
//
// The keys of a (stream, KV head) are cut into up to eight pieces, by the
// window alone, a CTA each; the pieces are one split, or more where a piece
// would pass 640 keys.  A CTA is a producer warp, which fills a ring of six
// 16 KB stages (16 bf16 keys or 32 e4m3 keys: one 3D TMA copy for K and one for
// V where a page holds them, else key by key with cp.async), and four consumer
// warps that compute S^T = K Q^T and O^T += V^T P^T with warp MMAs (8 query
// columns to an MMA, 16 a CTA; the tensor cores' 128-row tiles would stand
// nearly empty) with an online softmax per column, each warp on a tile and a
// column group of its own.  The tiles of a piece are dealt to two or four key
// slices; slices, pieces and splits merge in the order of the keys.
//
// A split's CTAs are a cluster that merges through distributed shared memory:
// one launch, no workspace.  Windows of several splits, and calls of more CTAs
// than the GPU holds where a cost model says so, run unclustered instead, a CTA
// on one or more pieces, and window_combine merges the pieces from the
// workspace.  Calls of many draft
// windows give a CTA 32 columns.  All of them round alike: a stream's bits do
// not depend on its batch.
//
// What bounds it: the bytes of K and V where there are many (64 streams of
// 4,096 bf16 keys: 539 MB in 85.7 us, 6.28 TB/s); whole waves of CTAs, two on
// an SM, and a tile's chain of latencies below that (32 streams of 4,096 e4m3
// keys: 137 MB in 36.7 us, 256 CTAs of two pieces on the 304 places); and for a
// few streams the host's call, the launch, the first tile's way in and the merge
// (one stream of 128 keys 6.6 us, four of 1,024 keys 8.2 us).  Two CTAs share an SM, so one
// streams while the other starts or merges.
#include <algorithm>
#include <cuda_fp16.h>

#include "pkv_dev.cuh"

namespace pkv {
namespace {

constexpr int kMaxCols = 32;                 // query columns of a (stream, KV head)
constexpr int kBlockCols = 16;               // ... of a CTA of small calls
constexpr int kMaxPieces = 8;                // pieces of a split
constexpr int kMaxSlices = 4;                // key slices of a piece
constexpr int kSplitKeys = 640;              // keys of a piece at most
constexpr int kMaxPages = kMaxPieces * kSplitKeys / 4 + 4;  // pages a CTA's run can touch
constexpr int kCtas = 304;                   // that the GPU holds at once, two an SM
// What a call of clusters costs against one of runs (CTAs on one to eight
// pieces each, merged by a second kernel), in keys of a wave of CTAs: a wave
// takes its CTAs' keys and kStartKeys (start, first tile, merge), and runs take
// kCombKeys more.  A run's keys count 9/10 where the bytes bound the call (a
// wave that is not full is faster) and 12/10 with CTAs of more than 16 columns
// and e4m3 pages of more than 8, which the latencies of a tile bound.  Measured,
// clusters against runs, those picked first: bf16, one token, windows of 4,096
// keys, 16 streams 23.9 us against 25.8; runs against clusters, 24 streams 36.6
// against 43.4, 64 streams 84.8 against 95.4; of 512 keys, 64 streams 24.4
// against 35.4; e4m3, 4,096 keys, 32 streams 37.4 against 40.1; with two tokens
// (16 columns) clusters against runs, 24 streams 50.7 against 55.6; bf16, four
// tokens (32 columns), 24 streams 69.7 against 72.0.
constexpr int kStartKeys = 300, kCombKeys = 100;
constexpr int kFreshGuard = 32;              // rows below the new tokens that a kernel just before may write
constexpr float kScaleLog2 = 0.0625f * 1.4426950408889634f;  // log2(e) / sqrt(256)

constexpr int kJoinBytes = 8192;             // O of a warp's 8 columns, in its registers' layout
constexpr int kPlane = 2048;                 // bf16: one 64-dim chunk of 16 rows

// Shapes of the two page formats' CTAs: four consumer warps, each on a tile (and
// column group) of its own with O over all dims in registers.  (Eight, a pair
// a tile with half the dims each, computed S twice and left 96 registers a
// thread: too few to load ahead of the MMAs, 2,100 cycles a tile.)
constexpr int kConsumers = 4;
template <bool kFp8>
struct Cfg {
    static constexpr int tile = kFp8 ? 32 : 16;                  // keys a stage
    static constexpr int half = 8192;                            // K or V bytes of a stage
    static constexpr int stage = 2 * half;
    static constexpr int slots = 6;
    static constexpr int bars = 2 * slots;                       // a tile's barriers: t % bars, its slot t % slots
    static_assert(half == tile * kHeadDim * (kFp8 ? 1 : 2), "whole rows");
    static constexpr int consumers = kConsumers;
    static constexpr int threads = consumers * 32 + 32;
    static constexpr int row = kFp8 ? kHeadDim + 12 : kHeadDim + 4;  // floats of a merge row
    static constexpr int off_scl = slots * stage;                // e4m3: 32 K and 32 V scales a stage
    static constexpr int off_page = off_scl + (kFp8 ? slots * 256 : 0);
    static constexpr int off_join = off_page + kMaxPages * 4;    // a piece's slices: 8 KB of O, then (m, l)
    static constexpr int off_join_ml = off_join + kJoinBytes;
    static constexpr int off_bar = off_join_ml + kMaxSlices * kBlockCols * 8;
    static constexpr int bytes = off_bar + 2 * bars * 8 + 16;
    static constexpr int smem = bytes + 1024;                    // with alignment slack
    // after the last tile the stages hold the merge rows, then the CTA's sum
    static constexpr int off_ml = 32 * row * 4;
    static constexpr int off_sum = (off_ml + 32 * 8 + 127) / 128 * 128;
    static constexpr int off_sum_ml = off_sum + kMaxCols * kHeadDim * 4;
    static_assert(off_sum_ml + kMaxCols * 8 <= slots * stage, "merge buffers reuse the stages");
    static_assert(off_join % 16 == 0 && off_bar % 8 == 0, "aligned");
};

struct WinArgs {
    const uint16_t *q;
    uint16_t *out;
    float *ws;
    float4 *stash;          // wide calls: a first pass's sums, kStash a CTA
    const uint16_t *k_new;  // fused store of the new tokens, or null
    const uint16_t *v_new;
    const uint16_t *ik_new;
    int32_t window, n_sink;
    int32_t pieces;     // pieces of a split
    int32_t run;        // pieces of a CTA; 0: one, and the split's CTAs are a cluster
    int32_t even;       // splits of each stream where all have as many, else 0
    int32_t even_cols;  // query columns (all KV heads) of each stream, likewise
};

// CTAs that share a (stream, KV head)'s columns.
__host__ __device__ inline int col_blocks(bool wide, int ncols) {
    const int block = wide ? kMaxCols : kBlockCols;
    return (ncols + block - 1) / block;
}
constexpr int kStash = kConsumers * 17 * 32;  // float4 a CTA: O and (m, l) of each lane

// Key slices of a piece: the tiles that a CTA of kBlockCols columns works on at
// once.  Each of a tile's barriers always belongs to one slice, which takes
// every phase of it: the slices divide their number.  (A slice that skipped a
// phase could not tell the tile before its own, not landed yet, from its own:
// both leave the same parity.)
__host__ __device__ inline int slices_of(int ncols) {
    const int ncg = ((ncols < kBlockCols ? ncols : kBlockCols) + 7) >> 3;
    return kConsumers / ncg;
}
static_assert(Cfg<false>::bars % kMaxSlices == 0 && Cfg<true>::bars % kMaxSlices == 0 && kConsumers == kMaxSlices,
              "1, 2 or 4 slices, each with barriers of its own");

// ---- cluster helpers ----------------------------------------------------------
__device__ __forceinline__ float4 peer_ld4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 peer_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

// The active consumer warps of a CTA meet (n threads).
__device__ __forceinline__ void join_sync(int n) {
    asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory");
}

// ---- small helpers --------------------------------------------------------------
__device__ __forceinline__ float max_rows(float v) {  // over the lanes that share lane & 3
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float sum_rows(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// Byte offset of 16-byte chunk c of row r inside a staged K or V tile, with the
// TMA's 128-byte swizzle.  bf16: four planes of 64 dims, each 16 rows x 128 B.
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return (c >> 3) * kPlane + r * 128 + ((((c & 7) ^ (r & 7))) << 4);
}
// e4m3: whole rows of 256 B, each two lines of 128 B.
__device__ __forceinline__ uint32_t swz8(int r, int c) {
    const int line = 2 * r + (c >> 3);
    return line * 128 + ((((c & 7) ^ (line & 7))) << 4);
}

// D (16x8 f32) += A (16x16 f16, row) B (16x8 f16, col).  Not volatile: it only
// reads its registers, and the compiler may place it among the conversions.
__device__ __forceinline__ void mma_half(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// s = 2^e x mant with mant in [1, 2); a zero or subnormal scale gives weight 0, one
// that is not finite gives NaN (its zero codes are NaN, and a row that holds an
// infinity has no other codes but NaN).
__device__ __forceinline__ void split_scale(float s, float &e, float &mant) {
    const uint32_t b = __float_as_uint(s);
    const int ex = static_cast<int>((b >> 23) & 0xffu);
    e = ex != 0 ? static_cast<float>(ex - 127) : -INFINITY;
    mant = ex == 0xff ? __uint_as_float(0x7fffffffu) : ex != 0 ? __uint_as_float((b & 0x007fffffu) | 0x3f800000u) : 0.f;
}

// ---- one CTA's run of keys --------------------------------------------------------
struct Run {
    WindowSpan sp;
    int s, kvh, split;
    int col0;              // its first query column
    int piece, n_pieces;   // its pieces of the split
    int key0, key1;        // their virtual keys
    int per;               // tiles of a piece
    int qbase;
    int sink_page, win_page, n_sink_pages, n_pages;  // the page list: sinks' pages, then the window's
};

template <int kTile, bool kWide>
__device__ __forceinline__ Run locate(const Common &c, const WinArgs &a) {
    Run u;
    u.n_pieces = max(1, a.run);
    const int per_split = a.pieces / u.n_pieces, b = static_cast<int>(blockIdx.x), item = b / per_split;
    // (a search through the streams' offsets costs a CTA of a full launch 1.5 us)
    u.s = a.even ? item / a.even : find_seq(c.n_seqs, item, [&](int t) { return c.seq[t].work_off; });
    const SeqDev &sd = c.seq[u.s];
    const int r = a.even ? item - u.s * a.even : item - sd.work_off;
    const int blocks = col_blocks(kWide, sd.ncols), q = r / blocks;
    u.col0 = (r - q * blocks) * kBlockCols;
    u.kvh = q / sd.nsplit;
    u.split = q - u.kvh * sd.nsplit;
    u.piece = (b - item * per_split) * u.n_pieces;
    u.sp = window_span(sd.len, sd.n_new, a.window, a.n_sink, kTile);
    u.per = sd.split_len / kTile;
    u.key0 = min(u.sp.nkeys, (u.split * a.pieces + u.piece) * sd.split_len);
    u.key1 = min(u.sp.nkeys, u.key0 + u.n_pieces * sd.split_len);
    u.qbase = sd.len - sd.n_new;
    u.sink_page = u.win_page = u.n_sink_pages = u.n_pages = 0;
    if (sd.table && u.key1 > u.key0) {
        if (u.key0 < u.sp.sink_end) {
            u.sink_page = u.key0 / sd.ptok;
            u.n_sink_pages = min(min(u.key1, u.sp.sink_end), a.n_sink) - 1;
            u.n_sink_pages = u.n_sink_pages / sd.ptok - u.sink_page + 1;
            u.n_pages = u.n_sink_pages;
        }
        if (u.key1 > u.sp.sink_end) {
            // the first seen position: the sinks may reach into the window's first tile
            int p0 = max(u.key0, u.sp.sink_end) + u.sp.shift;
            if (p0 >= a.n_sink) p0 = max(p0, u.sp.lo);
            const int p1 = u.key1 - 1 + u.sp.shift;
            u.win_page = p0 / sd.ptok;
            u.n_pages += p1 / sd.ptok - u.win_page + 1;
        }
    }
    return u;
}

// Position of virtual key v.
__device__ __forceinline__ int pos_of(const WindowSpan &sp, int v) {
    return v + (v >= sp.sink_end ? sp.shift : 0);
}

struct Ctx {
    uint8_t *stages;
    float *scl;          // e4m3: [slot][2][32] K then V scales
    int32_t *pages;      // ids of the run's pages (-1: outside the arena)
    uint64_t *full, *empty;
    volatile int *abort_flag;
};

// Where one staged key's rows come from (per lane; bf16: lanes 16.. repeat 0..15).
struct KeySrc {
    int pos;          // the position read
    int row;          // its row inside the page
    int64_t page;     // its page's offset (elements)
    bool seen;        // some query sees the key (else pos is a neighbour's)
    bool fresh;       // the row comes from the new tokens' input
    bool bad;         // its page id was outside the arena
};

template <int kTile>
__device__ __forceinline__ KeySrc key_src(const SeqDev &sd, const WinArgs &a, const Run &u, const Ctx &x,
                                          int v0, int lane) {
    KeySrc k;
    const int v = v0 + (lane & (kTile - 1));
    const int p = pos_of(u.sp, v);
    k.seen = v < u.key1 && (p < a.n_sink || p >= u.sp.lo);
    // the last position of the run, the last sink, or the window's first position
    k.pos = k.seen ? p : v >= u.key1 ? pos_of(u.sp, u.key1 - 1) : v < u.sp.sink_end ? a.n_sink - 1 : u.sp.lo;
    k.row = k.pos;
    k.page = 0;
    k.bad = false;
    if (sd.table) {
        const int page = k.pos / sd.ptok;
        k.row = k.pos - page * sd.ptok;
        const int id = x.pages[min(v, u.key1 - 1) < u.sp.sink_end ? page - u.sink_page
                                                                  : u.n_sink_pages + page - u.win_page];
        k.bad = id < 0;
        k.page = max(id, 0) * sd.ps;
    }
    k.fresh = a.k_new != nullptr && k.pos >= u.qbase;
    return k;
}

// Stage the bf16 tile of virtual keys v0 .. into `slot` key by key (the producer warp); the copies
// complete on `bar`, and new rows are stored into the cache too.
__device__ __forceinline__ void stage16(const Common &c, const WinArgs &a, const SeqDev &sd, const Run &u,
                                        const Ctx &x, int v0, int slot, uint64_t *bar, int lane, uint64_t pol) {
    const int H = c.n_kv_heads;
    const int64_t v_gap = (int64_t)H * sd.ptok * kHeadDim;  // V row - K row
    const KeySrc k = key_src<16>(sd, a, u, x, v0, lane);
    const int64_t krow = k.page + off_k(sd.ptok, u.kvh, k.row);
    uint8_t *kst = x.stages + slot * Cfg<false>::stage, *vst = kst + Cfg<false>::half;
    const uint16_t *ksrc, *vsrc;
    if (k.fresh) {
        const int64_t r = ((int64_t)sd.tok_off + (k.pos - u.qbase)) * H + u.kvh;
        ksrc = a.k_new + r * kHeadDim;
        vsrc = a.v_new + r * kHeadDim;
    } else {
        ksrc = sd.layer_base + krow;
        vsrc = ksrc + v_gap;
    }
    const int64_t kp = reinterpret_cast<int64_t>(ksrc), vp = reinterpret_cast<int64_t>(vsrc);
#pragma unroll 4
    for (int r = 0; r < 16; ++r) {
        const uint16_t *kr = reinterpret_cast<const uint16_t *>(shfl64(kp, r));
        const uint16_t *vr = reinterpret_cast<const uint16_t *>(shfl64(vp, r));
        cp_async16(kst + swz(r, lane), kr + lane * 8, pol);
        cp_async16(vst + swz(r, lane), vr + lane * 8, pol);
    }
    cp_async_mbar_arrive(bar);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    unsigned todo = __ballot_sync(0xffffffffu, k.fresh && k.seen && !k.bad && lane < 16 && u.col0 == 0);
    while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int p = __shfl_sync(0xffffffffu, k.pos, src), prow = __shfl_sync(0xffffffffu, k.row, src);
        const int64_t kr = shfl64(krow, src), pg = shfl64(k.page, src);
        const int64_t r = (int64_t)sd.tok_off + (p - u.qbase);
        uint16_t *dst = const_cast<uint16_t *>(sd.layer_base) + kr;
        const uint4 kv = __ldg(reinterpret_cast<const uint4 *>(a.k_new + (r * H + u.kvh) * kHeadDim) + lane);
        const uint4 vv = __ldg(reinterpret_cast<const uint4 *>(a.v_new + (r * H + u.kvh) * kHeadDim) + lane);
        reinterpret_cast<uint4 *>(dst)[lane] = kv;
        reinterpret_cast<uint4 *>(dst + v_gap)[lane] = vv;
        if (u.kvh == 0 && a.ik_new != nullptr && lane < c.idx_dim / 8) {
            // the indexer-key row of the same position, written once (KV head 0)
            uint16_t *idst = const_cast<uint16_t *>(sd.layer_base) + pg + off_ik(H, c.idx_dim, sd.ptok, prow);
            reinterpret_cast<uint4 *>(idst)[lane] =
                __ldg(reinterpret_cast<const uint4 *>(a.ik_new + r * c.idx_dim) + lane);
        }
    }
}

// The same for e4m3 pages: 32 code rows of K and V and their scales.  New rows
// are quantized here (the rule of pkv_store) into the stage and the cache.
__device__ __forceinline__ void stage8(const Common &c, const WinArgs &a, const SeqDev &sd, const Run &u,
                                       const Ctx &x, int v0, int slot, uint64_t *bar, int lane, uint64_t pol) {
    const int H = c.n_kv_heads;
    const KeySrc k = key_src<32>(sd, a, u, x, v0, lane);
    const uint8_t *base = reinterpret_cast<const uint8_t *>(sd.layer_base);
    const int64_t pg = 2 * k.page;
    const int64_t kc = pg + off8_code(false, H, sd.ptok, u.kvh, k.row);
    const int64_t vc = pg + off8_code(true, H, sd.ptok, u.kvh, k.row);
    uint8_t *st = x.stages + slot * Cfg<true>::stage;
    uint8_t *sc = reinterpret_cast<uint8_t *>(x.scl) + slot * 256;
    constexpr int kCodes = Cfg<true>::half;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int item = lane + 32 * i, rr = item >> 4, ch = item & 15;
        const int64_t krr = shfl64(kc, rr), vrr = shfl64(vc, rr);
        if (!__shfl_sync(0xffffffffu, k.fresh, rr)) {
            cp_async16(st + swz8(rr, ch), base + krr + 16 * ch, pol);
            cp_async16(st + kCodes + swz8(rr, ch), base + vrr + 16 * ch, pol);
        }
    }
    if (!k.fresh) {
        cp_async4(sc + 4 * lane, base + pg + off8_scale(false, H, sd.ptok, u.kvh, k.row));
        cp_async4(sc + 128 + 4 * lane, base + pg + off8_scale(true, H, sd.ptok, u.kvh, k.row));
    }
    // rows whose source is a new token: quantized by the whole warp, one at a
    // time; one that no query sees only needs finite codes
    unsigned todo = __ballot_sync(0xffffffffu, k.fresh);
    while (todo) {
        const int rr = __ffs(todo) - 1;
        todo &= todo - 1;
        const bool seen = __shfl_sync(0xffffffffu, k.seen, rr);
        if (!seen) {
#pragma unroll
            for (int v = 0; v < 2; ++v)
                *reinterpret_cast<uint2 *>(st + v * kCodes + swz8(rr, lane >> 1) + (lane & 1) * 8) = make_uint2(0u, 0u);
            if (lane < 2) reinterpret_cast<float *>(sc)[32 * lane + rr] = 0.f;
            continue;
        }
        const int p = __shfl_sync(0xffffffffu, k.pos, rr), row = __shfl_sync(0xffffffffu, k.row, rr);
        const bool write = u.col0 == 0 && !__shfl_sync(0xffffffffu, k.bad, rr);
        const int64_t pg_rr = shfl64(pg, rr);
        const int64_t tr = (int64_t)sd.tok_off + (p - u.qbase);  // its packed input row
        const bool ik_row = write && u.kvh == 0 && a.ik_new != nullptr && lane < c.idx_dim / 8;
        const uint4 in_k = __ldg(reinterpret_cast<const uint4 *>(a.k_new + (tr * H + u.kvh) * kHeadDim) + lane);
        const uint4 in_v = __ldg(reinterpret_cast<const uint4 *>(a.v_new + (tr * H + u.kvh) * kHeadDim) + lane);
        const uint4 in_ik = ik_row ? __ldg(reinterpret_cast<const uint4 *>(a.ik_new + tr * c.idx_dim) + lane)
                                   : make_uint4(0u, 0u, 0u, 0u);
        uint8_t *lb = const_cast<uint8_t *>(base) + pg_rr;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint2 codes;
            const float scale = quantize_row8(v ? in_v : in_k, &codes);
            *reinterpret_cast<uint2 *>(st + v * kCodes + swz8(rr, lane >> 1) + (lane & 1) * 8) = codes;
            if (lane == 0) reinterpret_cast<float *>(sc)[32 * v + rr] = scale;
            if (write) {
                *reinterpret_cast<uint2 *>(lb + off8_code(v, H, sd.ptok, u.kvh, row) + 8 * lane) = codes;
                if (lane == 0) *reinterpret_cast<float *>(lb + off8_scale(v, H, sd.ptok, u.kvh, row)) = scale;
            }
        }
        if (ik_row)
            reinterpret_cast<uint4 *>(lb + 2 * off_ik_f(true, H, c.idx_dim, sd.ptok, row))[lane] = in_ik;
    }
    cp_async_mbar_arrive(bar);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// One query column's softmax over some keys: maximum, sum, and O of four dims.
struct Sum {
    float m, l;
    float4 o;
};

// The sum over n partials in order (a piece's slices, a split's pieces);
// ml_of(k) and acc_of(k) load partial k.
template <int kMax, typename FM, typename FO>
__device__ __forceinline__ Sum merge_parts(int n, FM ml_of, FO acc_of) {
    float2 ml[kMax];
    float4 v[kMax];
#pragma unroll
    for (int k = 0; k < kMax; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < n) {
            ml[k] = ml_of(k);
            v[k] = acc_of(k);
        }
    }
    Sum r;
    r.m = -INFINITY;
    r.l = 0.f;
    r.o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kMax; ++k) r.m = fmaxf(r.m, ml[k].x);
#pragma unroll
    for (int k = 0; k < kMax; ++k) {
        const float w = r.m == -INFINITY ? 0.f : ex2(ml[k].x - r.m);
        // fused explicitly: both kernels that merge round alike
        r.l = fmaf(w, ml[k].y, r.l);
        r.o.x = fmaf(w, v[k].x, r.o.x);
        r.o.y = fmaf(w, v[k].y, r.o.y);
        r.o.z = fmaf(w, v[k].z, r.o.z);
        r.o.w = fmaf(w, v[k].w, r.o.w);
    }
    return r;
}

// Four dims of an output row.  A query sees its own position at least, so l is
// 0 only where every score is -infinity: NaN then, as where a score or a row that
// is read is NaN.
__device__ __forceinline__ void write_out(uint16_t *out, const Sum &r) {
    uint2 pk;
    pk.x = pack_bf16(__fdiv_rn(r.o.x, r.l), __fdiv_rn(r.o.y, r.l));
    pk.y = pack_bf16(__fdiv_rn(r.o.z, r.l), __fdiv_rn(r.o.w, r.l));
    *reinterpret_cast<uint2 *>(out) = pk;
}

// Whether the query at position p (-1: a padding column) sees position kp.
__device__ __forceinline__ bool sees(int p, int kp, int window, int n_sink) {
    return kp <= p && (kp > p - window || kp < n_sink);
}

template <bool kFp8, bool kRuns, bool kWide>
__global__ void __launch_bounds__(Cfg<kFp8>::threads, 2)
    window_partial(const __grid_constant__ Common c, const __grid_constant__ DecodeMaps maps,
                   const __grid_constant__ WinArgs a) {
    using F = Cfg<kFp8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctx x;
    x.stages = smem;
    x.scl = reinterpret_cast<float *>(smem + F::off_scl);
    x.pages = reinterpret_cast<int32_t *>(smem + F::off_page);
    x.full = reinterpret_cast<uint64_t *>(smem + F::off_bar);
    x.empty = x.full + F::bars;
    x.abort_flag = reinterpret_cast<volatile int *>(x.empty + F::bars);
    constexpr int S = F::slots, B = F::bars;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Run u = locate<F::tile, kWide>(c, a);
    const SeqDev &sd = c.seq[u.s];
    const int ncols = sd.ncols, G = c.group, H = c.n_kv_heads;
    const int nc = min(ncols - u.col0, kWide ? kMaxCols : kBlockCols);  // this CTA's columns
    const int ncg = (nc + 7) >> 3;                   // in groups of 8
    // A piece's tile t belongs to key slice t % slices.  A CTA takes all slices
    // at once, ks_n tiles in its warps together, or (more than kBlockCols
    // columns) one slice after the other in two passes.  A piece takes whole
    // rounds of the slices: empty tiles fill its last one.
    const int slices = slices_of(ncols);
    const int passes = kWide && ncols > kBlockCols ? 2 : 1, ks_n = passes == 1 ? slices : 1;
    const int round = (u.per + slices - 1) / slices * slices;  // a piece's tiles, empty ones among them
    const int pass_tiles = passes == 1 ? round : round / 2;
    const int ntiles = kRuns || u.key1 > u.key0 ? u.n_pieces * round : 0;
    const int cg = warp % ncg, ks = warp / ncg;
    const bool active = warp < F::consumers && ks < ks_n;

    if (tid == 0) {
        for (int i = 0; i < B; ++i) {
            mbar_init(&x.full[i], 1);
            mbar_init(&x.empty[i], ncg);
        }
        *x.abort_flag = 0;
        fence_mbar_init();
    }
    for (int j = tid; j < u.n_pages; j += F::threads) {
        const int p = j < u.n_sink_pages ? u.sink_page + j : u.win_page + (j - u.n_sink_pages);
        // small pages between the sinks and the window may lie inside one tile:
        // no row of theirs is read
        if ((int64_t)p * sd.ptok >= a.n_sink && (int64_t)(p + 1) * sd.ptok <= u.sp.lo) continue;
        const int id = __ldg(sd.table + p);
        const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(sd.n_pages);
        if (!ok && c.status) atomicOr(c.status, PKV_DEV_BAD_PAGE);
        x.pages[j] = ok ? id : -1;
    }
    __syncthreads();

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[16][4];  // O^T: 16 tiles of 16 dims, this lane's two columns
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    int issued = 0;  // tiles the producer has staged
    if (warp == F::consumers) {
        // ---------------- producer ----------------
        const uint64_t pol = policy_evict_first();
        const void *map = sd.tma >= 0 ? &maps.map[sd.tma] : nullptr;
        const int v_rows = H * sd.ptok;       // map rows from a K row to its V row
        const bool wide = window_wide(sd);    // e4m3: a copy takes the tile's 32 rows, else 16
        // cached rows more than kFreshGuard below the new tokens do not depend
        // on the previous kernel: their tiles stream before the wait
        const int early_end = u.qbase - kFreshGuard;
        bool waited = false;
        int first = -1;         // lane i: first virtual key of tile t0 + i, -1: an empty tile
        int yk = -1, yk2 = 0;   // map rows of its first K row and its 17th, -1: not runs of cached rows
        int64_t sc = 0, sc2 = 0;  // e4m3: byte offsets of those rows' K scales
        for (int t = 0; t < ntiles; ++t, ++issued) {
            if ((t & 31) == 0) {
                // the next 32 tiles' rows, a tile a lane: looked up one by one
                // they would take the warp longer than a tile takes to arrive
                const int w = (t + lane) / pass_tiles, j = t + lane - w * pass_tiles;
                const int pc = passes == 1 ? w : w >> 1, tp = passes == 1 ? j : 2 * j + (w & 1);
                const int v0 = u.key0 + (pc * u.per + tp) * F::tile, p0 = pos_of(u.sp, v0);
                first = tp < u.per && v0 < u.key1 ? v0 : -1;
                yk = -1;
                if (map != nullptr && first >= 0 && v0 + F::tile <= u.key1 &&
                    (p0 >= u.sp.lo || p0 + F::tile <= a.n_sink || a.n_sink >= u.sp.lo) &&
                    (a.k_new == nullptr || p0 + F::tile <= u.qbase)) {
                    auto look = [&](int p, int &y, int64_t &scale) {
                        int row = p;
                        int64_t pg = 0;
                        if (sd.table) {
                            const int page = p / sd.ptok;
                            row = p - page * sd.ptok;
                            const int id = x.pages[v0 < u.sp.sink_end ? page - u.sink_page : u.n_sink_pages + page - u.win_page];
                            pg = max(id, 0) * sd.ps;  // (-1 was reported when it was looked up)
                        }
                        if constexpr (kFp8) {
                            y = static_cast<int>(sd.layer_row + (2 * pg + off8_code(false, H, sd.ptok, u.kvh, row)) / kHeadDim);
                            scale = 2 * pg + off8_scale(false, H, sd.ptok, u.kvh, row);
                        } else {
                            y = static_cast<int>(sd.layer_row + (pg + off_k(sd.ptok, u.kvh, row)) / kHeadDim);
                        }
                    };
                    look(p0, yk, sc);
                    if (kFp8 && !wide) look(p0 + 16, yk2, sc2);
                }
            }
            const int slot = t % S, y = __shfl_sync(0xffffffffu, yk, t & 31);
            const int v0 = __shfl_sync(0xffffffffu, first, t & 31);
            uint64_t *const bar = &x.full[t % B];
            if (t >= S) {
                if (!__all_sync(0xffffffffu, mbar_wait(&x.empty[(t - S) % B], ((t - S) / B) & 1, c.status))) {
                    *x.abort_flag = 1;
                    break;
                }
                fence_proxy_async_smem();  // the slot's last reads come before the next tile's writes
            }
            if (v0 < 0) {
                if (lane == 0) mbar_arrive(bar);
                continue;
            }
            if (!waited && pos_of(u.sp, v0) + F::tile > early_end) {
                pdl_wait();
                waited = true;
            }
            if (y >= 0) {
                // a page holds the keys (e4m3: or a page each of their halves): a
                // copy of K and one of V, and with e4m3 pages of their scales
                uint8_t *const kst = x.stages + slot * F::stage;
                const int64_t s0 = kFp8 ? shfl64(sc, t & 31) : 0, s1 = kFp8 && !wide ? shfl64(sc2, t & 31) : 0;
                const int y2 = kFp8 && !wide ? __shfl_sync(0xffffffffu, yk2, t & 31) : 0;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, F::stage + (kFp8 ? 256 : 0));
                    if constexpr (kFp8) {
                        const uint8_t *base = reinterpret_cast<const uint8_t *>(sd.layer_base);
                        float *const scl = x.scl + slot * 64;
                        tma_load_3d(kst, map, 0, 0, y, bar, pol);
                        tma_load_3d(kst + F::half, map, 0, 0, y + v_rows, bar, pol);
                        bulk_g2s(scl, base + s0, wide ? 128 : 64, bar, pol);
                        bulk_g2s(scl + 32, base + s0 + 4 * (int64_t)v_rows, wide ? 128 : 64, bar, pol);
                        if (!wide) {
                            tma_load_3d(kst + F::half / 2, map, 0, 0, y2, bar, pol);
                            tma_load_3d(kst + F::half + F::half / 2, map, 0, 0, y2 + v_rows, bar, pol);
                            bulk_g2s(scl + 16, base + s1, 64, bar, pol);
                            bulk_g2s(scl + 48, base + s1 + 4 * (int64_t)v_rows, 64, bar, pol);
                        }
                    } else {
                        tma_load_3d(kst, map, 0, y, 0, bar, pol);
                        tma_load_3d(kst + F::half, map, 0, y + v_rows, 0, bar, pol);
                    }
                }
            } else if constexpr (kFp8) {
                stage8(c, a, sd, u, x, v0, slot, bar, lane, pol);
            } else {
                stage16(c, a, sd, u, x, v0, slot, bar, lane, pol);
            }
            __syncwarp();
        }
        if (!waited) pdl_wait();
    } else if (active) {
        // ---------------- consumers ----------------
        const int g = lane >> 2, c4 = lane & 3;
        const int bcol = u.col0 + cg * 8 + g;
        const uint16_t *qr = nullptr;
        if (bcol < ncols) {
            const int j = bcol / G;
            qr = a.q + (((int64_t)sd.tok_off + j) * c.n_q_heads + u.kvh * G + (bcol - j * G)) * kHeadDim;
        }
        asm volatile("" ::"l"(qr));
        pdl_wait();
        // The next kernel may start: the kernel before this one is done, and of
        // what this one writes a decode reads no row before its own wait (none
        // within kFreshGuard of its new tokens).  Let go before the wait, calls
        // of 32 new tokens could have read rows of the last call but one.
        if (tid == 0) pdl_trigger();
        uint32_t qf[16][2];
        float qs0, qs1;  // e4m3: what a score of this lane's two columns is scaled by
        if constexpr (kFp8) {
            // dims 64 c4 .. 64 c4 + 63 of the row, converted to f16 once.  bf16 has
            // the wider range: a power of two first takes the row's largest element
            // to 2^14 .. 2^15, exactly, and goes into the scores' scale
            uint4 w[8];
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = qr ? __ldg(reinterpret_cast<const uint4 *>(qr + 64 * c4) + i) : make_uint4(0u, 0u, 0u, 0u);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                             __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu)));
            }
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = static_cast<int>(max(top >> 16, top & 0xffffu) >> 7);  // biased exponent
            // (zeros, and rows with an infinity or NaN, stay as they are)
            const int e = ex == 0 || ex == 0xff ? 0 : max(ex - 127 - 14, -100);
            const float dn = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            const float up = kScaleLog2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            qs0 = __shfl_sync(0xffffffffu, up, 8 * c4);
            qs1 = __shfl_sync(0xffffffffu, up, 8 * c4 + 4);
            const auto pair = [&](uint32_t x) { return bits_of(__floats2half2_rn(dn * bf16_lo(x), dn * bf16_hi(x))); };
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                qf[2 * i][0] = pair(w[i].x);
                qf[2 * i][1] = pair(w[i].y);
                qf[2 * i + 1][0] = pair(w[i].z);
                qf[2 * i + 1][1] = pair(w[i].w);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) {
                const int d = kk * 16 + 2 * c4;
                qf[kk][0] = qr ? __ldg(reinterpret_cast<const uint32_t *>(qr + d)) : 0u;
                qf[kk][1] = qr ? __ldg(reinterpret_cast<const uint32_t *>(qr + d + 8)) : 0u;
            }
        }
        // the positions of this lane's two columns (-1: padding)
        const int c0 = u.col0 + cg * 8 + 2 * c4;
        const int p0 = c0 < ncols ? u.qbase + c0 / G : -1;
        const int p1 = c0 + 1 < ncols ? u.qbase + (c0 + 1) / G : -1;
        const uint32_t s_base = smem_u32(x.stages);
        const int kr_ = (lane & 7) + 8 * ((lane >> 3) & 1), kcb = lane >> 4;
        const int vr_ = (lane & 7) + 8 * (lane >> 4), vcb = (lane >> 3) & 1;
        float uo[2] = {-INFINITY, -INFINITY};  // e4m3: O's own reference (logit + V-scale exponent)

        auto reset = [&] {
            m[0] = m[1] = uo[0] = uo[1] = -INFINITY;
            l[0] = l[1] = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        };
        // The sums of a piece (or of a slice of it, in two passes) are complete:
        // l over the key rows, O on the logits' maximum.  They stay in registers for the cluster's merge, or the
        // piece's slices join into slice 0's (as merge_parts would), which go
        // to the workspace, O [piece of the unit][column][256], then (m, l),
        // and the next piece starts anew.  The slices hand O over lane by lane,
        // 8 KB at a time; written out one by one they are two to four times
        // the traffic (64 streams of 4,096 keys 99.0 us against 92.3).
        auto finish_pass = [&](int pc, int pass) {
            l[0] = sum_rows(l[0]);
            l[1] = sum_rows(l[1]);
            if constexpr (kFp8) {
                const float f0 = uo[0] == -INFINITY ? 0.f : ex2(uo[0] - m[0]);
                const float f1 = uo[1] == -INFINITY ? 0.f : ex2(uo[1] - m[1]);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    acc[i][0] *= f0;
                    acc[i][1] *= f1;
                    acc[i][2] *= f0;
                    acc[i][3] *= f1;
                }
            }
            if (kWide && passes > 1) {
                // slice 0's sums wait in the workspace for slice 1's, each lane its own
                float4 *const st = a.stash + (int64_t)blockIdx.x * kStash + warp * (17 * 32) + lane;
                if (pass == 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) st[i * 32] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                    st[16 * 32] = make_float4(m[0], l[0], m[1], l[1]);
                    reset();
                    return;
                }
                const float4 ml = st[16 * 32];
                const float M0 = fmaxf(ml.x, m[0]), M1 = fmaxf(ml.z, m[1]);
                const float w0 = M0 == -INFINITY ? 0.f : ex2(ml.x - M0), w1 = M1 == -INFINITY ? 0.f : ex2(ml.z - M1);
                const float x0 = M0 == -INFINITY ? 0.f : ex2(m[0] - M0), x1 = M1 == -INFINITY ? 0.f : ex2(m[1] - M1);
                l[0] = fmaf(x0, l[0], fmaf(w0, ml.y, 0.f));
                l[1] = fmaf(x1, l[1], fmaf(w1, ml.w, 0.f));
                m[0] = M0;
                m[1] = M1;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 v = st[i * 32];
                    acc[i][0] = fmaf(x0, acc[i][0], fmaf(w0, v.x, 0.f));
                    acc[i][1] = fmaf(x1, acc[i][1], fmaf(w1, v.y, 0.f));
                    acc[i][2] = fmaf(x0, acc[i][2], fmaf(w0, v.z, 0.f));
                    acc[i][3] = fmaf(x1, acc[i][3], fmaf(w1, v.w, 0.f));
                }
            }
            if constexpr (!kRuns) return;
            if (!kWide || ks_n > 1) {
                const int cl = cg * 8 + 2 * c4;  // this lane's first column in the CTA
                float4 *const jml = reinterpret_cast<float4 *>(smem + F::off_join_ml);  // [slice][two columns]
                float4 *const jo = reinterpret_cast<float4 *>(smem + F::off_join) + cg * 8 * 32 + lane;
                if (g == 0) jml[(ks * kBlockCols + cl) / 2] = make_float4(m[0], l[0], m[1], l[1]);
                join_sync(ncg * ks_n * 32);
                if (ks == 0) {
                    const float4 own = make_float4(m[0], l[0], m[1], l[1]);
                    for (int k = 1; k < ks_n; ++k) {
                        const float4 ml = jml[(k * kBlockCols + cl) / 2];
                        m[0] = fmaxf(m[0], ml.x);
                        m[1] = fmaxf(m[1], ml.z);
                    }
                    const float w0 = m[0] == -INFINITY ? 0.f : ex2(own.x - m[0]);
                    const float w1 = m[1] == -INFINITY ? 0.f : ex2(own.z - m[1]);
                    l[0] = fmaf(w0, own.y, 0.f);
                    l[1] = fmaf(w1, own.w, 0.f);
    #pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        acc[i][0] = fmaf(w0, acc[i][0], 0.f);
                        acc[i][1] = fmaf(w1, acc[i][1], 0.f);
                        acc[i][2] = fmaf(w0, acc[i][2], 0.f);
                        acc[i][3] = fmaf(w1, acc[i][3], 0.f);
                    }
                }
                for (int k = 1; k < ks_n; ++k) {
                    float w0 = 0.f, w1 = 0.f;
                    if (ks == 0) {
                        const float4 ml = jml[(k * kBlockCols + cl) / 2];
                        w0 = m[0] == -INFINITY ? 0.f : ex2(ml.x - m[0]);
                        w1 = m[1] == -INFINITY ? 0.f : ex2(ml.z - m[1]);
                        l[0] = fmaf(w0, ml.y, l[0]);
                        l[1] = fmaf(w1, ml.w, l[1]);
                    }
    #pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 8 tiles of 16 dims at a time
                        if (k > 1 || h > 0) join_sync(ncg * ks_n * 32);  // the part before has been read
                        if (ks == k) {
    #pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float(&t)[4] = acc[8 * h + i];
                                jo[i * 32] = make_float4(t[0], t[1], t[2], t[3]);
                            }
                        }
                        join_sync(ncg * ks_n * 32);
                        if (ks == 0) {
    #pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 v = jo[i * 32];
                                float(&t)[4] = acc[8 * h + i];
                                t[0] = fmaf(w0, v.x, t[0]);
                                t[1] = fmaf(w1, v.y, t[1]);
                                t[2] = fmaf(w0, v.z, t[2]);
                                t[3] = fmaf(w1, v.w, t[3]);
                            }
                        }
                    }
                }
            }
            if (ks == 0) {
                const int64_t n_part = (int64_t)sd.nsplit * a.pieces;  // of a unit
                const int64_t part = u.kvh * n_part + u.split * a.pieces + u.piece + pc;
                float *o = a.ws + sd.ws_off + (part * ncols + c0) * kHeadDim;
                float *ml = a.ws + sd.ws_off + (int64_t)H * n_part * ncols * kHeadDim + (part * ncols + c0) * 2;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (c0 + e < ncols) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if constexpr (kFp8) {
                                *reinterpret_cast<float2 *>(o + e * kHeadDim + 32 * g + 2 * i) =
                                    make_float2(acc[i][e], acc[i][e + 2]);
                            } else {
                                o[e * kHeadDim + 16 * i + g] = acc[i][e];
                                o[e * kHeadDim + 16 * i + g + 8] = acc[i][e + 2];
                            }
                        }
                        if (g == 0) *reinterpret_cast<float2 *>(ml + 2 * e) = make_float2(m[e], l[e]);
                    }
                }
            }
            reset();
        };

        const int n_pieces = kRuns ? u.n_pieces : ntiles > 0 ? 1 : 0;
        bool ok = true;
        // (after a wait that ran out the warp still meets the others at each piece's end)
        for (int w = 0; w < n_pieces * passes; ++w) {
            const int pc = passes == 1 ? w : w >> 1, pass = w - pc * passes;
            for (int tp = pass + ks; ok && tp < round; tp += slices) {
                const int t = w * pass_tiles + (passes == 1 ? tp : tp >> 1), slot = t % S;
                ok = __all_sync(0xffffffffu, mbar_wait(&x.full[t % B], (t / B) & 1, c.status));
                if (!ok) {
                    *x.abort_flag = 1;
                    break;
                }
                const int v0 = u.key0 + (pc * u.per + tp) * F::tile;
                if (tp >= u.per || v0 >= u.key1) {
                    if (lane == 0) mbar_arrive(&x.empty[t % B]);
                    continue;
                }
                const uint8_t *const st = x.stages + slot * F::stage;
                const float *const scl = x.scl + slot * 64;  // e4m3
                // S^T of the tile's keys and this lane's two columns: rows g and g + 8
                // of each 16 keys, in log2 units, -inf where the column's query does
                // not see the key
                constexpr int kSub = F::tile / 16;
                float sx[kSub][4];
#pragma unroll
                for (int u16 = 0; u16 < kSub; ++u16) {
                    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (kFp8) {
                        // two accumulator chains, a quarter of the dims at a time
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 w0 = *reinterpret_cast<const uint4 *>(st + swz8(16 * u16 + g, 4 * c4 + i));
                            const uint4 w1 = *reinterpret_cast<const uint4 *>(st + swz8(16 * u16 + g + 8, 4 * c4 + i));
                            uint32_t z[4][4];
                            f16_of_codes(w0.x, z[0][0], z[0][2]);
                            f16_of_codes(w1.x, z[0][1], z[0][3]);
                            f16_of_codes(w0.y, z[1][0], z[1][2]);
                            f16_of_codes(w1.y, z[1][1], z[1][3]);
                            f16_of_codes(w0.z, z[2][0], z[2][2]);
                            f16_of_codes(w1.z, z[2][1], z[2][3]);
                            f16_of_codes(w0.w, z[3][0], z[3][2]);
                            f16_of_codes(w1.w, z[3][1], z[3][3]);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_half((j & 1) ? sb : sa, z[j][0], z[j][1], z[j][2], z[j][3], qf[4 * i + j][0],
                                         qf[4 * i + j][1]);
                        }
                        const float ka_scl = scl[16 * u16 + g], kb_scl = scl[16 * u16 + g + 8];
                        sa[0] = (sa[0] + sb[0]) * ka_scl * qs0;
                        sa[1] = (sa[1] + sb[1]) * ka_scl * qs1;
                        sa[2] = (sa[2] + sb[2]) * kb_scl * qs0;
                        sa[3] = (sa[3] + sb[3]) * kb_scl * qs1;
                    } else {
                        // two accumulator chains, four K fragments loaded before their MMAs
                        const uint32_t kbs = s_base + slot * F::stage;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t f[4][4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                ldsm_x4(kbs + h * kPlane + swz(kr_, 2 * j + kcb), f[j][0], f[j][1], f[j][2], f[j][3]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t(&x4)[4] = f[j];
                                mma_bf16((j & 1) ? sb : sa, x4[0], x4[1], x4[2], x4[3], qf[4 * h + j][0], qf[4 * h + j][1]);
                            }
                        }
                    }
                    const int ka = pos_of(u.sp, v0) + 16 * u16 + g, kb = ka + 8;
                    const auto score = [&](int i) { return kFp8 ? sa[i] : (sa[i] + sb[i]) * kScaleLog2; };
                    sx[u16][0] = sees(p0, ka, a.window, a.n_sink) ? score(0) : -INFINITY;
                    sx[u16][1] = sees(p1, ka, a.window, a.n_sink) ? score(1) : -INFINITY;
                    sx[u16][2] = sees(p0, kb, a.window, a.n_sink) ? score(2) : -INFINITY;
                    sx[u16][3] = sees(p1, kb, a.window, a.n_sink) ? score(3) : -INFINITY;
                }
                // online softmax of the two columns
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int u16 = 0; u16 < kSub; ++u16) {
                    t0 = fmaxf(t0, fmaxf(sx[u16][0], sx[u16][2]));
                    t1 = fmaxf(t1, fmaxf(sx[u16][1], sx[u16][3]));
                }
                const float n0 = fmaxf(m[0], max_rows(t0)), n1 = fmaxf(m[1], max_rows(t1));
                const float o0 = n0 == -INFINITY ? 0.f : n0, o1 = n1 == -INFINITY ? 0.f : n1;
                const float al0 = ex2(m[0] - o0), al1 = ex2(m[1] - o1);  // 0 while nothing was summed
                m[0] = n0;
                m[1] = n1;
                l[0] *= al0;
                l[1] *= al1;
                // the weights of O, as two parts (hi + lo) in the MMAs' B layout
                uint32_t wh[kSub][2], wl[kSub][2];
                float be0 = al0, be1 = al1;  // what O is rescaled by
                if constexpr (kFp8) {
                    // a V scale 2^E x mant goes into the key's weight, with a running
                    // maximum of logit + E as O's reference: weights in [0, 2), split
                    // into f16 hi + lo parts (about 22 significant bits)
                    float e[kSub][2], mt[kSub][2], r0 = -INFINITY, r1 = -INFINITY;
#pragma unroll
                    for (int u16 = 0; u16 < kSub; ++u16) {
                        split_scale(scl[32 + 16 * u16 + g], e[u16][0], mt[u16][0]);
                        split_scale(scl[32 + 16 * u16 + g + 8], e[u16][1], mt[u16][1]);
                        l[0] += ex2(sx[u16][0] - o0) + ex2(sx[u16][2] - o0);
                        l[1] += ex2(sx[u16][1] - o1) + ex2(sx[u16][3] - o1);
                        r0 = fmaxf(r0, fmaxf(sx[u16][0] + e[u16][0], sx[u16][2] + e[u16][1]));
                        r1 = fmaxf(r1, fmaxf(sx[u16][1] + e[u16][0], sx[u16][3] + e[u16][1]));
                    }
                    const float nu0 = fmaxf(uo[0], max_rows(r0)), nu1 = fmaxf(uo[1], max_rows(r1));
                    const float z0 = nu0 == -INFINITY ? 0.f : nu0, z1 = nu1 == -INFINITY ? 0.f : nu1;
                    be0 = ex2(uo[0] - z0);
                    be1 = ex2(uo[1] - z1);
                    uo[0] = nu0;
                    uo[1] = nu1;
#pragma unroll
                    for (int u16 = 0; u16 < kSub; ++u16) {
                        const float q0 = ex2(sx[u16][0] + e[u16][0] - z0) * mt[u16][0];
                        const float q1 = ex2(sx[u16][1] + e[u16][0] - z1) * mt[u16][0];
                        const float q2 = ex2(sx[u16][2] + e[u16][1] - z0) * mt[u16][1];
                        const float q3 = ex2(sx[u16][3] + e[u16][1] - z1) * mt[u16][1];
                        const __half2 h01 = __floats2half2_rn(q0, q1), h23 = __floats2half2_rn(q2, q3);
                        const __half2 l01 = __floats2half2_rn(q0 - __low2float(h01), q1 - __high2float(h01));
                        const __half2 l23 = __floats2half2_rn(q2 - __low2float(h23), q3 - __high2float(h23));
                        wh[u16][0] = movmatrix_t(bits_of(h01));
                        wh[u16][1] = movmatrix_t(bits_of(h23));
                        wl[u16][0] = movmatrix_t(bits_of(l01));
                        wl[u16][1] = movmatrix_t(bits_of(l23));
                    }
                } else {
                    // P as a bf16 pair hi + lo (lo = p - hi exactly): about 16
                    // significant bits of the weights reach the float32 accumulator
                    const float e0 = ex2(sx[0][0] - o0), e1 = ex2(sx[0][1] - o1);
                    const float e2 = ex2(sx[0][2] - o0), e3 = ex2(sx[0][3] - o1);
                    l[0] += e0 + e2;
                    l[1] += e1 + e3;
                    const uint32_t h01 = pack_bf16(e0, e1), h23 = pack_bf16(e2, e3);
                    wh[0][0] = movmatrix_t(h01);
                    wh[0][1] = movmatrix_t(h23);
                    wl[0][0] = movmatrix_t(pack_bf16(e0 - bf16_lo(h01), e1 - bf16_hi(h01)));
                    wl[0][1] = movmatrix_t(pack_bf16(e2 - bf16_lo(h23), e3 - bf16_hi(h23)));
                }
                if (__any_sync(0xffffffffu, be0 != 1.f || be1 != 1.f)) {  // some reference grew
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        acc[i][0] *= be0;
                        acc[i][1] *= be1;
                        acc[i][2] *= be0;
                        acc[i][3] *= be1;
                    }
                }
                // O^T += V^T P^T
                if constexpr (kFp8) {
#pragma unroll
                    for (int u16 = 0; u16 < kSub; ++u16) {
                        // V codes of keys 2c, 2c+1, 2c+8, 2c+9, dims 32g .. 32g+31
                        uint32_t w[4][8];
                        const uint8_t *vb = st + F::half;
                        const int kr[4] = {2 * c4, 2 * c4 + 1, 2 * c4 + 8, 2 * c4 + 9};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 z0 = *reinterpret_cast<const uint4 *>(vb + swz8(16 * u16 + kr[i], 2 * g));
                            const uint4 z1 = *reinterpret_cast<const uint4 *>(vb + swz8(16 * u16 + kr[i], 2 * g + 1));
                            w[i][0] = z0.x;
                            w[i][1] = z0.y;
                            w[i][2] = z0.z;
                            w[i][3] = z0.w;
                            w[i][4] = z1.x;
                            w[i][5] = z1.y;
                            w[i][6] = z1.z;
                            w[i][7] = z1.w;
                        }
                        // four dim tiles at a time: a hi and a lo product of one
                        // tile follow each other at the MMA's latency
#pragma unroll
                        for (int i4 = 0; i4 < 16; i4 += 4) {
                            uint32_t z[4][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                // codes of dims 32g + 2 (i4 + i) and + 1: {key, next key}
                                // of the first dim, then of the second
                                const int wi = (i4 + i) >> 1, b = 2 * (i & 1);
                                const uint32_t sel = b | ((4 + b) << 4) | ((b + 1) << 8) | ((5 + b) << 12);
                                f16_of_codes(__byte_perm(w[0][wi], w[1][wi], sel), z[i][0], z[i][1]);
                                f16_of_codes(__byte_perm(w[2][wi], w[3][wi], sel), z[i][2], z[i][3]);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_half(acc[i4 + i], z[i][0], z[i][1], z[i][2], z[i][3], wh[u16][0], wh[u16][1]);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_half(acc[i4 + i], z[i][0], z[i][1], z[i][2], z[i][3], wl[u16][0], wl[u16][1]);
                        }
                    }
                } else {
                    const uint32_t vbs = s_base + slot * F::stage + F::half;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t f[4][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            ldsm_x4_t(vbs + h * kPlane + swz(vr_, 2 * j + vcb), f[j][0], f[j][1], f[j][2], f[j][3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t(&x4)[4] = f[j];
                            mma_bf16(acc[4 * h + j], x4[0], x4[1], x4[2], x4[3], wh[0][0], wh[0][1]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t(&x4)[4] = f[j];
                            mma_bf16(acc[4 * h + j], x4[0], x4[1], x4[2], x4[3], wl[0][0], wl[0][1]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.empty[t % B]);
            }
            finish_pass(pc, pass);
        }
    }
    __syncthreads();  // every staged tile is consumed (or the CTA gave up)
    const bool failed = *x.abort_flag != 0;
    // after a wait that ran out, every copy issued lands before the memory goes
    if (failed)
        for (int j = max(0, issued - S); j < issued; ++j) mbar_wait(&x.full[j % B], (j / B) & 1, nullptr);
    if (kRuns) return;  // the slices are joined; window_combine merges the pieces

    // ---- merge the CTA's key slices, in order ----
    const int NC = ncg * 8;
    float *mbuf = reinterpret_cast<float *>(x.stages);               // [ks][NC][row]
    float *mlb = reinterpret_cast<float *>(x.stages + F::off_ml);    // [ks][NC][2]
    float *sum = reinterpret_cast<float *>(x.stages + F::off_sum);   // [nc][256]
    float *sum_ml = reinterpret_cast<float *>(x.stages + F::off_sum_ml);
    if (active && !failed) {
        const int g = lane >> 2, c0 = cg * 8 + 2 * (lane & 3);
        float *b0 = mbuf + (ks * NC + c0) * F::row, *b1 = b0 + F::row;
        if constexpr (kFp8) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = 33 * g + 2 * i;  // dim 32 g + 2 i, skewed by g against bank conflicts
                b0[d] = acc[i][0];
                b1[d] = acc[i][1];
                b0[d + 1] = acc[i][2];
                b1[d + 1] = acc[i][3];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = 16 * i + g;
                b0[d] = acc[i][0];
                b1[d] = acc[i][1];
                b0[d + 8] = acc[i][2];
                b1[d + 8] = acc[i][3];
            }
        }
        if (g == 0) {
            float *ml = mlb + (ks * NC + c0) * 2;
            ml[0] = m[0];
            ml[1] = l[0];
            ml[2] = m[1];
            ml[3] = l[1];
        }
    }
    __syncthreads();
    for (int idx = tid; idx < nc * (kHeadDim / 4); idx += F::threads) {
        const int col = idx / (kHeadDim / 4), d = 4 * (idx - col * (kHeadDim / 4));
        const int ds = kFp8 ? d + (d >> 5) : d;
        const Sum r = merge_parts<kMaxSlices>(
            ks_n, [&](int k) { return *reinterpret_cast<const float2 *>(mlb + (k * NC + col) * 2); },
            [&](int k) {
                const float *v = mbuf + (k * NC + col) * F::row + ds;
                return make_float4(v[0], v[1], v[2], v[3]);
            });
        *reinterpret_cast<float4 *>(sum + col * kHeadDim + d) = r.o;
        if (d == 0) *reinterpret_cast<float2 *>(sum_ml + 2 * col) = make_float2(r.m, r.l);
    }
    // ---- then the cluster's CTAs, in order ----
    cluster_sync();
    if (!failed) {
        for (int idx = u.piece * F::threads + tid; idx < nc * (kHeadDim / 4); idx += a.pieces * F::threads) {
            const int col = idx / (kHeadDim / 4), d = 4 * (idx - col * (kHeadDim / 4));
            const Sum r = merge_parts<kMaxPieces>(
                a.pieces, [&](int k) { return peer_ld2(peer_addr(sum_ml + 2 * col, k)); },
                [&](int k) { return peer_ld4(peer_addr(sum + col * kHeadDim + d, k)); });
            const int j = (u.col0 + col) / G, h = u.col0 + col - j * G;
            write_out(a.out + (((int64_t)sd.tok_off + j) * c.n_q_heads + u.kvh * G + h) * kHeadDim + d, r);
        }
    }
    cluster_sync();  // the peers have read this CTA's sums
}

// Merge of the pieces' partials for calls whose CTAs are not clustered: a CTA a
// query column, a thread four dims; the split's pieces and the splits in order,
// as a cluster merges its CTAs' sums.  A thread loads all pieces of a split
// together, and a CTA is small (no shared memory, two warps) so that it can
// start beside the last partial CTAs.
constexpr int kCombThreads = kHeadDim / 4;
__global__ void __launch_bounds__(kCombThreads)
    window_combine(const __grid_constant__ Common c, const __grid_constant__ WinArgs a) {
    pdl_trigger();  // the next kernel waits for this grid before it reads what it writes
    const int i = static_cast<int>(blockIdx.x);
    const int s = a.even_cols ? i / a.even_cols : find_seq(c.n_seqs, i, [&](int t) { return c.seq[t].comb_off; });
    const SeqDev &sd = c.seq[s];
    const int r = a.even_cols ? i - s * a.even_cols : i - sd.comb_off;
    const int ncols = sd.ncols, unit = r / ncols, col = r - unit * ncols, G = c.group;
    const int d = 4 * static_cast<int>(threadIdx.x), j = col / G;
    const int64_t n_part = (int64_t)sd.nsplit * a.pieces;
    const float *acc = a.ws + sd.ws_off + (unit * n_part * ncols + col) * kHeadDim + d;
    const float *ml = a.ws + sd.ws_off + (int64_t)c.n_kv_heads * n_part * ncols * kHeadDim + (unit * n_part * ncols + col) * 2;
    uint16_t *out = a.out + (((int64_t)sd.tok_off + j) * c.n_q_heads + unit * G + (col - j * G)) * kHeadDim + d;
    asm volatile("" ::"l"(acc), "l"(ml), "l"(out));
    pdl_wait();
    Sum t;
    for (int sp = 0; sp < sd.nsplit; ++sp) {
        const int64_t p0 = (int64_t)sp * a.pieces;
        const Sum x = merge_parts<kMaxPieces>(
            a.pieces, [&](int p) { return __ldcg(reinterpret_cast<const float2 *>(ml + (p0 + p) * ncols * 2)); },
            [&](int p) { return __ldcg(reinterpret_cast<const float4 *>(acc + (p0 + p) * ncols * kHeadDim)); });
        if (sp == 0) {
            t = x;
        } else {
            const float M = fmaxf(t.m, x.m);
            const float wt = M == -INFINITY ? 0.f : ex2(t.m - M), wx = M == -INFINITY ? 0.f : ex2(x.m - M);
            t.l = wt * t.l + wx * x.l;
            t.o.x = wt * t.o.x + wx * x.o.x;
            t.o.y = wt * t.o.y + wx * x.o.y;
            t.o.z = wt * t.o.z + wx * x.o.z;
            t.o.w = wt * t.o.w + wx * x.o.w;
            t.m = M;
        }
    }
    write_out(out, t);
}

using WindowKernel = void (*)(Common, DecodeMaps, WinArgs);
template <bool kFp8>
WindowKernel window_kernel_of(bool runs, bool wide) {
    return runs ? (wide ? window_partial<kFp8, true, true> : window_partial<kFp8, true, false>)
                : (wide ? window_partial<kFp8, false, true> : window_partial<kFp8, false, false>);
}
WindowKernel window_kernel(bool fp8, bool runs, bool wide) {
    return fp8 ? window_kernel_of<true>(runs, wide) : window_kernel_of<false>(runs, wide);
}

}  // namespace

// Pieces of a split, by the window alone (a stream's bits must not depend on
// its batch): 128 keys a piece before there is another.
static int window_pieces(int32_t window, int32_t n_sink) {
    const int64_t keys = (int64_t)window + n_sink + 32;
    int n = 1;
    while (n < kMaxPieces && keys > 128 * n) n *= 2;
    return n;
}

// The most virtual keys of a stream of up to `len` positions and n_new new
// tokens.  The count itself goes up and down by a tile with the length (the
// window starts anywhere in its first tile), this never goes down: splits by it
// need no more workspace for a shorter stream.
static int64_t most_keys(int32_t len, int32_t n_new, int32_t window, int32_t n_sink, int32_t tile) {
    const int64_t sinks = ((int64_t)n_sink + tile - 1) / tile * tile;
    return std::min<int64_t>(len, sinks + ((int64_t)window + n_new - 1) + (tile - 1));
}

// Splits only where a piece could pass kSplitKeys keys.  A call of streams with
// more than kBlockCols columns gives each kBlockCols a CTA while the CTAs fit
// the GPU at once, else all of them one: the bits are the same.  Four draft
// tokens of 8 heads, windows of 2,047 keys, 16 columns a CTA against 32: 8
// streams 15.4 us against 21.7, 16 streams (512 CTAs against 256) 30.9 against
// 25.0, 64 streams (which read twice the bytes from L2) 118 against 100.5.
int plan_window(Common &c, int32_t window, int32_t n_sink, WindowPlan *plan) {
    const int pieces = window_pieces(window, n_sink);
    const int tile = c.kv_fp8 ? Cfg<true>::tile : Cfg<false>::tile;
    bool split = false, wide = false, over8 = false;
    int64_t items = 0, cols = 0, floats = 0, keys = 0;
    for (int s = 0; s < c.n_seqs; ++s) {
        SeqDev &d = c.seq[s];
        if ((int64_t)d.n_new * c.group > kMaxCols) return PKV_EINVAL;
        d.ncols = d.n_new * c.group;
        d.nsplit = 1;
        d.split_len = tile;
        if (d.ncols == 0) continue;
        const WindowSpan sp = window_span(d.len, d.n_new, window, n_sink, tile);
        d.nsplit = static_cast<int32_t>((most_keys(d.len, d.n_new, window, n_sink, tile) - 1) / (pieces * kSplitKeys) + 1);
        const int per = (sp.nkeys - 1) / (d.nsplit * pieces) + 1;  // keys of a piece
        d.split_len = (per + tile - 1) / tile * tile;
        split |= d.nsplit > 1;
        wide |= d.ncols > kBlockCols;
        over8 |= d.ncols > 8;
        items += (int64_t)c.n_kv_heads * d.nsplit * col_blocks(false, d.ncols);
    }
    const bool many = items * pieces > kCtas;
    wide = wide && many;
    items = 0;
    for (int s = 0; s < c.n_seqs; ++s) {
        SeqDev &d = c.seq[s];
        d.work_off = static_cast<int32_t>(items);
        d.comb_off = static_cast<int32_t>(cols);
        d.ws_off = floats;
        if (d.ncols == 0) continue;
        items += (int64_t)c.n_kv_heads * d.nsplit * col_blocks(wide, d.ncols);
        cols += (int64_t)c.n_kv_heads * d.ncols;
        keys += (int64_t)c.n_kv_heads * col_blocks(wide, d.ncols) * window_span(d.len, d.n_new, window, n_sink, tile).nkeys;
        floats += (int64_t)c.n_kv_heads * d.nsplit * pieces * d.ncols * (kHeadDim + 2);
        floats = (floats + 63) / 64 * 64;
    }
    if (items * pieces > INT32_MAX) return PKV_EINVAL;
    const bool some = pieces > 1 && (split || many);  // calls that may run as runs of pieces
    // the least cost: a cluster a split, or runs of pieces (which have to merge splits)
    const int64_t per = items ? keys / (items * pieces) : 0;  // keys of a piece
    const auto waves = [&](int run) { return (items * pieces / run + kCtas - 1) / kCtas; };
    int64_t best = split ? INT64_MAX : waves(1) * (per + kStartKeys) * 10;
    plan->run = 0;
    for (int run = 1; some && run <= pieces; run *= 2) {
        const int64_t cost = waves(run) * (run * per * (wide || (c.kv_fp8 && over8) ? 12 : 9) + kStartKeys * 10) + kCombKeys * 10;
        if (cost < best) {
            best = cost;
            plan->run = run;
        }
    }
    const bool combine = plan->run > 0;
    plan->cost = best;
    plan->keys = keys;
    plan->items = static_cast<int32_t>(items);
    plan->comb = combine ? static_cast<int32_t>(cols) : 0;
    plan->pieces = pieces;
    plan->wide = wide;
    plan->ctas = static_cast<int32_t>(items * (pieces / std::max(1, plan->run)));
    // sized for either kind of call, so that the size for a stream's longest
    // length and most new tokens covers every shorter one and fewer
    plan->stash_off = some ? floats : 0;
    plan->ws_bytes = static_cast<size_t>(plan->stash_off) * 4 +
                     (wide ? static_cast<size_t>(items * pieces) * kStash * sizeof(float4) : 0);
    return PKV_OK;
}

int launch_window(const Common &c, const WindowPlan &plan, const DecodeMaps &maps, int32_t window,
                  int32_t n_sink, const uint16_t *q, uint16_t *out, float *ws, const uint16_t *k_new,
                  const uint16_t *v_new, const uint16_t *ik_new, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    if (once_per_device(attr_done, [] {
            for (int i = 0; i < 8; ++i) {
                const void *fn = reinterpret_cast<const void *>(window_kernel(i & 1, i & 2, i & 4));
                const int bytes = i & 1 ? Cfg<true>::smem : Cfg<false>::smem;
                if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
                    return PKV_ECUDA;
                if (cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared) != cudaSuccess)
                    return PKV_ECUDA;
            }
            // an SM left with a small carveout could not take a CTA of the next call
            return cuda_rc(cudaFuncSetAttribute(window_combine, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                cudaSharedmemCarveoutMaxShared));
        }) != PKV_OK)
        return PKV_ECUDA;
    WinArgs a{q, out, ws, reinterpret_cast<float4 *>(ws + plan.stash_off), k_new, v_new, ik_new, window, n_sink,
              plan.pieces, plan.run, 0, 0};
    if (plan.items % c.n_seqs == 0) a.even = plan.items / c.n_seqs;
    if (plan.comb % c.n_seqs == 0) a.even_cols = plan.comb / c.n_seqs;
    for (int s = 0; s < c.n_seqs; ++s) {
        if (c.seq[s].work_off != s * a.even) a.even = 0;
        if (c.seq[s].comb_off != s * a.even_cols) a.even_cols = 0;
    }
    const bool clustered = plan.run == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.ctas));
    cfg.blockDim = dim3(c.kv_fp8 ? Cfg<true>::threads : Cfg<false>::threads);
    cfg.dynamicSmemBytes = c.kv_fp8 ? Cfg<true>::smem : Cfg<false>::smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = clustered ? a.pieces : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto *const fn = window_kernel(c.kv_fp8 != 0, !clustered, plan.wide);
    if (cudaLaunchKernelEx(&cfg, fn, c, maps, a) != cudaSuccess)
        return PKV_ECUDA;
    if (clustered) return PKV_OK;
    return launch_status(
        launch_pdl(window_combine, static_cast<unsigned>(plan.comb), kCombThreads, 0, stream, c, a));
}

}  // namespace pkv
