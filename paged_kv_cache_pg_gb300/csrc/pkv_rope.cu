// Rotary positions: rows rotated by their tokens' positions, alone
// (pkv_rope_rows) or on the way into the pages (pkv_rope_store).
//
// Pair i of a row at position p turns by p f_i.  The frequencies come as
// fractions of a turn times 2^64, so p times one, modulo 2^64, is that product
// without its whole turns, exactly (the frequency itself is a float64's: 2^-22 of a
// turn at most at a position of 2^31); its top 32 bits (a signed fraction of a half
// turn) go to sincospif.  In float32 radians a
// position of 10^6 would leave 0.03 of the fastest pair's angle to chance.
//
// A small call has a CTA a token.  A large one is cut into units of up to four
// tokens, and as many CTAs as the GPU holds take every so many-th, the next unit's
// rows on their way while one's are turned: a prompt of 8,192 tokens of 16 query and
// 2 KV heads (172 MB) takes 31.7 us, 80 % of the copy rate (CTAs of a unit each took
// 1.2 us longer, units of 48 KB and two CTAs an SM 3.8).  What is left: the first
// rows' way in and the last ones' way out, and 7 units of 6.7 a CTA.  A
// unit's tokens' streams, pages and rows are found once, by a thread a token (the
// streams' first tokens lie together in the launch parameters: read from the
// streams' own records, 64 of them took 6 us of a call), and their cosines and sines
// computed once, into shared memory, for all of their heads (16 query rows and 2 key
// rows use the same 32 to 128 pairs); a small call's, with positions from the launch
// parameters, before the grid-dependency wait.  Rows come by bulk copies: held in
// registers, two rows a warp in flight, a prompt took 47 us.  A warp takes a row of
// 256 elements (two of 128) at a time, a lane 16 bytes of it and, with
// PKV_ROPE_HALF, the 16 bytes of its pairs' other elements.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pkv_dev.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kBlockTokens = 4;  // of a unit of large calls
constexpr int kSegHeads = 64;    // query heads of a unit
constexpr int kStageBytes = 24 * 1024;  // of a unit of several tokens
constexpr int kSmBytes = 228 * 1024, kStaticBytes = 7 * 1024, kCtas = 4;  // of an SM, of a CTA besides its stages, CTAs of an SM

// Cosine and sine of position p at one pair's frequency, times the scale.
__device__ __forceinline__ float2 turn(uint64_t turns, int32_t p, float scale) {
    const uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(p));
    const float x = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ void widen(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
}
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// How a rope's pairs lie in a lane's 16 bytes of a row (chunk ch), known when
// compiled: pairs inside it; their other elements 16 bytes of the same row; or
// (rot_dim, or half of it, not a multiple of 8) anywhere.
enum Mode { kStill, kInside, kApart, kAnyhow };
int mode_of(const pkv_rope &r) {
    return r.pairs == PKV_ROPE_INTERLEAVED ? (r.rot_dim % 8 == 0 ? kInside : kAnyhow) : (r.rot_dim % 16 == 0 ? kApart : kAnyhow);
}

// A lane's part in turning a token's rows: its elements' cosines, and the sines
// with the sign they take, in registers over all of the token's rows.
template <int kMode>
struct Turner {
    float c[8], s[8];
    int ch, other, rot, inter;
    bool on;  // some of its elements turn

    __device__ __forceinline__ Turner(const float2 *cs, int chunk, const pkv_rope &r) {
        ch = chunk;
        rot = r.rot_dim;
        inter = r.pairs;
        const int half = rot >> 1, e0 = 8 * ch;
        on = kMode != kStill && e0 < rot;
        other = e0 < half ? ch + (half >> 3) : ch - (half >> 3);
        if (!on) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = e0 + e;
            const bool first = kMode == kInside || (kMode == kAnyhow && inter) ? !(e & 1) : i < half;
            const int pair = kMode == kInside || (kMode == kAnyhow && inter) ? i >> 1 : first ? i : i - half;
            const float2 w = kMode != kAnyhow || i < rot ? cs[pair] : make_float2(1.f, 0.f);
            c[e] = w.x;
            s[e] = first ? -w.y : w.y;
        }
    }
    // Its elements of a row (in shared memory), turned, as float32.
    __device__ __forceinline__ void turn_row(const uint16_t *row, float (&x)[8]) const {
        widen(*(reinterpret_cast<const uint4 *>(row) + ch), x);
        if (!on) return;
        float y[8];
        if constexpr (kMode == kApart) {
            widen(*(reinterpret_cast<const uint4 *>(row) + other), y);
        } else if constexpr (kMode == kInside) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
            const int half = rot >> 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * ch + e, j = inter ? i ^ 1 : i < half ? i + half : i - half;
                y[e] = i < rot ? __uint_as_float(static_cast<uint32_t>(row[j]) << 16) : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (kMode != kAnyhow || 8 * ch + e < rot) x[e] = x[e] * c[e] + y[e] * s[e];
    }
};

// The streams' first tokens, and how the launch is cut.
struct RopeTokens {
    int32_t tok_off[PKV_MAX_SEQS];
    int32_t total, block;  // tokens, and those of a unit
    int32_t segs;          // units of a token: kSegHeads query heads each
    int32_t bytes;         // of a token's rows in shared memory
    int32_t units, ctas;
};
// What a CTA works on at a time.
struct RopeUnit {
    int32_t tok0;
    int n, seg;  // tokens; which of their heads
    __device__ __forceinline__ RopeUnit(const RopeTokens &tk, int u) {
        const int group = u / tk.segs;
        seg = u - group * tk.segs;
        tok0 = group * tk.block;
        n = min(tk.block, tk.total - tok0);
    }
};
// A CTA's token as its rows need it.
struct TokenAt {
    uint16_t *page;     // its page of the layer, or null (outside the arena)
    int32_t row, ptok;  // its row there, positions of a page
    int32_t pos;        // what its rows turn by
};

// Stream of a token, found by one thread.
__device__ __forceinline__ int stream_of(const Common &c, const RopeTokens &tk, int32_t tok) {
    return find_seq(c.n_seqs, tok, [&](int t) { return tk.tok_off[t]; });
}

// The cosines and sines of n tokens: a thread a pair, as many tokens at once as
// that leaves threads for.
struct Filler {
    int pair, first, step;  // this thread's pair, its first token, and from one to the next (none: first >= kThreads)
    __device__ __forceinline__ explicit Filler(int pairs) {
        step = kThreads / pairs;
        first = threadIdx.x / pairs;
        pair = threadIdx.x - first * pairs;
        if (first >= step) first = kThreads;
    }
    __device__ __forceinline__ void operator()(const uint64_t *turns, float scale, const TokenAt *at, int n, float2 *cs) const {
        for (int k = first; k < n; k += step) cs[k * kMaxPairs + pair] = turn(turns[pair], at[k].pos, scale);
    }
};
// The frequencies of the launch parameters, each by one thread, into shared memory:
// read where they are, a warp's 32 different ones were as many reads one after the
// other for every token (the prompt 32.8 us, 4,096 tokens' indexer queries 8.4 for
// 7.4).
__device__ __forceinline__ void copy_turns(const pkv_rope &rope, uint64_t *turns) {
    if (threadIdx.x < rope.rot_dim >> 1) {
        uint64_t v;
        asm volatile("ld.u64 %0, [%1];" : "=l"(v) : "l"(rope.turns + threadIdx.x));
        turns[threadIdx.x] = v;
    }
}

// A CTA's way through its units, every tk.ctas-th: the next one's rows come while
// this one's are turned.  load(unit, stage) and place(unit, places) start a unit's
// copies (by the first warp) and find its tokens; rows(unit, stage) turns them.
template <bool kTurns, typename Load, typename Place, typename Rows>
__device__ __forceinline__ void through_units(const pkv_rope &rope, const RopeTokens &tk, bool pos_given, bool early,
                                              uint64_t (&full)[2], TokenAt (&at)[2][kBlockTokens], uint64_t *turns, float2 *cs, uint32_t *status,
                                              const Load &load, const Place &place, const Rows &rows) {
    if (threadIdx.x == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        fence_mbar_init();
    }
    int u = blockIdx.x;
    RopeUnit now(tk, u), next = now;
    if (kTurns) copy_turns(rope, turns);
    const Filler fill(kTurns ? rope.rot_dim >> 1 : kMaxPairs);
    if (pos_given) pdl_wait();
    place(now, at[0]);
    __syncthreads();
    const bool before = kTurns && !pos_given && tk.block == 1;  // a small call's turns, beside the kernel before
    if (before) fill(turns, rope.scale, at[0], now.n, cs);
    pdl_wait();
    if (early && threadIdx.x == 0) pdl_trigger();
    load(now, 0);
    u += tk.ctas;
    bool more = u < tk.units;
    if (more) {
        next = RopeUnit(tk, u);
        load(next, 1);
        place(next, at[1]);
    }
    for (int it = 0;; ++it) {
        const int s = it & 1;
        if (kTurns && !(before && it == 0)) fill(turns, rope.scale, at[s], now.n, cs);
        __syncthreads();
        const bool there = mbar_wait(&full[s], (it >> 1) & 1, status);
        if (there) rows(now, s);
        // Where a wait ran out no barrier is used again, and what is on its way lands
        // (or another limit passes) before the memory goes
        if (!more) {
            if (!there) mbar_wait(&full[s], (it >> 1) & 1, nullptr);
            return;
        }
        if (__syncthreads_or(!there)) {  // (the stage, its places and the turns are done with)
            mbar_wait(&full[s], (it >> 1) & 1, nullptr);
            mbar_wait(&full[s ^ 1], ((it + 1) >> 1) & 1, nullptr);
            return;
        }
        now = next;
        u += tk.ctas;
        more = u < tk.units;
        if (more) {
            next = RopeUnit(tk, u);
            load(next, s);
            place(next, at[s]);
        }
    }
}

// Rows of kDim elements, c.n_q_heads a token.
template <int kDim, int kMode>
__global__ void __launch_bounds__(kThreads, kCtas)
    rope_rows(const __grid_constant__ Common c, const __grid_constant__ pkv_rope rope, const __grid_constant__ RopeRows r,
              const __grid_constant__ RopeTokens tk) {
    extern __shared__ __align__(16) uint8_t smem[];  // one or two stages of each token's rows
    __shared__ __align__(16) float2 cs[kBlockTokens * kMaxPairs];
    __shared__ uint64_t turns[kMaxPairs];
    __shared__ TokenAt at[2][kBlockTokens];
    __shared__ uint64_t full[2];
    constexpr int kChunks = kDim / 8, kRowsWarp = 32 / kChunks;
    const int stage_bytes = tk.block * tk.bytes;
    const auto heads_of = [&](const RopeUnit &u) { return min(kSegHeads, c.n_q_heads - u.seg * kSegHeads); };
    const auto load = [&](const RopeUnit &u, int stage) {
        if (threadIdx.x) return;
        const uint64_t pol = policy_evict_first();
        const int bytes = heads_of(u) * kDim * 2;
        mbar_arrive_expect_tx(&full[stage], u.n * bytes);
        for (int k = 0; k < u.n; ++k)
            bulk_g2s(smem + stage * stage_bytes + k * tk.bytes, r.q + (u.tok0 + k) * r.q_stride + (int64_t)u.seg * kSegHeads * kDim, bytes,
                     &full[stage], pol);
    };
    const auto place = [&](const RopeUnit &u, TokenAt *to) {
        if (threadIdx.x >= u.n) return;
        const int tok = u.tok0 + threadIdx.x;
        if (r.pos) {
            to[threadIdx.x].pos = __ldg(r.pos + tok);
        } else {
            const int s = stream_of(c, tk, tok);
            to[threadIdx.x].pos = c.seq[s].len - c.seq[s].n_new + (tok - tk.tok_off[s]);
        }
    };
    const int lane = threadIdx.x & 31, ch = lane % kChunks, sub = lane / kChunks, ways = kWarps / tk.block;
    const int warp = threadIdx.x >> 5, k = warp / ways, first = warp - k * ways;
    const auto rows = [&](const RopeUnit &u, int stage) {
        if (k >= u.n) return;
        const Turner<kMode> t(cs + k * kMaxPairs, ch, rope);
        const uint16_t *const src = reinterpret_cast<const uint16_t *>(smem + stage * stage_bytes + k * tk.bytes);
        uint16_t *const dst = r.q_out + (u.tok0 + k) * r.q_out_stride + (int64_t)u.seg * kSegHeads * kDim;
        for (int h = first * kRowsWarp + sub; h < heads_of(u); h += ways * kRowsWarp) {
            float x[8];
            t.turn_row(src + h * kDim, x);
            *(reinterpret_cast<uint4 *>(dst + h * kDim) + ch) = narrow(x);
        }
    };
    // (nothing here is read before a grid-dependency wait: the next kernel may start)
    through_units<true>(rope, tk, r.pos != nullptr, true, full, at, turns, cs, c.status, load, place, rows);
}

// A token's rows: its queries (when given), keys, values, indexer row.  kStill:
// the keys are stored as they are (and there are no queries).  early: the next
// kernel may start once all older ones are done, before the rows are there.
template <bool kFp8, int kMode>
__global__ void __launch_bounds__(kThreads, kCtas)
    rope_store(const __grid_constant__ Common c, const __grid_constant__ pkv_rope rope, const __grid_constant__ RopeRows r,
               const __grid_constant__ RopeTokens tk, bool early) {
    extern __shared__ __align__(16) uint8_t smem[];  // one or two stages of each token's queries, K and V heads, indexer row
    __shared__ __align__(16) float2 cs[kMode != kStill ? kBlockTokens * kMaxPairs : 1];
    __shared__ uint64_t turns[kMode != kStill ? kMaxPairs : 1];
    __shared__ TokenAt at[2][kBlockTokens];
    __shared__ uint64_t full[2];
    const int stage_bytes = tk.block * tk.bytes, H = c.n_kv_heads;
    const auto queries = [&](const RopeUnit &u) { return kMode != kStill && r.q ? min(kSegHeads, c.n_q_heads - u.seg * kSegHeads) : 0; };
    const auto load = [&](const RopeUnit &u, int stage) {
        if (threadIdx.x >= 32) return;
        const uint64_t pol = policy_evict_first();
        const int q = queries(u) * kHeadDim * 2, kv = u.seg == 0 ? H * kHeadDim * 2 : 0, ik = u.seg == 0 ? c.idx_dim * 2 : 0;  // bytes
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&full[stage], u.n * (q + 2 * kv + ik));
        __syncwarp();
        const int k = threadIdx.x >> 2, part = threadIdx.x & 3;  // four parts a token
        if (k < u.n) {
            const int64_t tok = u.tok0 + k;
            uint8_t *const to = smem + stage * stage_bytes + k * tk.bytes;
            if (part == 0 && q) bulk_g2s(to, r.q + tok * r.q_stride + (int64_t)u.seg * kSegHeads * kHeadDim, q, &full[stage], pol);
            if (part == 1 && kv) bulk_g2s(to + q, r.k + tok * r.k_stride, kv, &full[stage], pol);
            if (part == 2 && kv) bulk_g2s(to + q + kv, r.v + tok * r.v_stride, kv, &full[stage], pol);
            if (part == 3 && ik) bulk_g2s(to + q + 2 * kv, r.ik + tok * r.ik_stride, ik, &full[stage], pol);
        }
    };
    const auto place = [&](const RopeUnit &u, TokenAt *to) {
        if (threadIdx.x >= u.n) return;
        const int tok = u.tok0 + threadIdx.x, s = stream_of(c, tk, tok);
        const SeqDev &sd = c.seq[s];
        TokenAt t;
        const int32_t place = sd.len - sd.n_new + (tok - tk.tok_off[s]);
        t.ptok = sd.ptok;
        t.pos = r.pos ? __ldg(r.pos + tok) : place;
        t.page = const_cast<uint16_t *>(sd.layer_base);
        t.row = place;
        if (sd.table && u.seg == 0) {
            const int32_t p = place / sd.ptok, id = __ldg(sd.table + p);
            t.row = place - p * sd.ptok;
            if (static_cast<uint32_t>(id) < static_cast<uint32_t>(sd.n_pages)) {
                t.page += (int64_t)id * sd.ps;
            } else {
                t.page = nullptr;
                if (c.status) atomicOr(c.status, PKV_DEV_BAD_PAGE);
            }
        }
        to[threadIdx.x] = t;
    };
    // a CTA's warps share its tokens out: eight, or fewer, to each, which take its rows in turn
    const int lane = threadIdx.x & 31, ways = kWarps / tk.block, warp = threadIdx.x >> 5, k = warp / ways, first = warp - k * ways;
    const auto rows = [&](const RopeUnit &u, int stage) {
        if (k >= u.n) return;
        const int nq = queries(u), nkv = u.seg == 0 ? 2 * H : 0;
        const bool idx = u.seg == 0 && c.idx_dim;
        const Turner<kMode> t(cs + (kMode != kStill ? k * kMaxPairs : 0), lane, rope);
        const TokenAt place = at[stage][k];
        const uint16_t *const src = reinterpret_cast<const uint16_t *>(smem + stage * stage_bytes + k * tk.bytes);
        uint16_t *const dst = r.q_out + (u.tok0 + k) * r.q_out_stride + (int64_t)u.seg * kSegHeads * kHeadDim;
        uint8_t *const b8 = reinterpret_cast<uint8_t *>(place.page);
        for (int i = first; i < nq + nkv + (idx ? 1 : 0); i += ways) {
            const uint16_t *const row = src + i * kHeadDim;
            if (i < nq) {
                float x[8];
                t.turn_row(row, x);
                *(reinterpret_cast<uint4 *>(dst + i * kHeadDim) + lane) = narrow(x);
                continue;
            }
            if (!place.page) break;
            const bool v = i >= nq + H;
            const int head = i - nq - (v ? H : 0);
            if (i == nq + nkv) {
                if (lane < kIdxDim / 8)
                    *(reinterpret_cast<uint4 *>(place.page + off_ik_f(kFp8, H, c.idx_dim, place.ptok, place.row)) + lane) =
                        *(reinterpret_cast<const uint4 *>(row) + lane);
            } else if constexpr (kFp8) {
                float x[8];
                if (v || kMode == kStill) widen(*(reinterpret_cast<const uint4 *>(row) + lane), x);
                else t.turn_row(row, x);
                uint2 codes;
                const float scale = quantize_row8f(x, &codes);
                *reinterpret_cast<uint2 *>(b8 + off8_code(v, H, place.ptok, head, place.row) + lane * 8) = codes;
                if (lane == 0) *reinterpret_cast<float *>(b8 + off8_scale(v, H, place.ptok, head, place.row)) = scale;
            } else {
                uint4 o = *(reinterpret_cast<const uint4 *>(row) + lane);
                if (!v && kMode != kStill) {
                    float x[8];
                    t.turn_row(row, x);
                    o = narrow(x);
                }
                *(reinterpret_cast<uint4 *>(place.page + (v ? off_v(H, place.ptok, head, place.row) : off_k(place.ptok, head, place.row))) + lane) = o;
            }
        }
    };
    through_units<kMode != kStill>(rope, tk, r.pos != nullptr, early, full, at, turns, cs, c.status, load, place, rows);
    pdl_trigger_after_writes();  // the next decode may read these rows early
}

bool to_turns(double radians, uint64_t *out) {
    if (!std::isfinite(radians)) return false;
    double t = radians / 6.283185307179586476925286766559;
    t -= std::floor(t);
    if (!(t >= 0.0 && t < 1.0)) t = 0.0;  // (a tiny negative one rounds up to a whole turn)
    *out = static_cast<uint64_t>(std::ldexp(t, 64));
    return true;
}

bool rope_shape_ok(int32_t rot_dim, int32_t pairs, const void *out) {
    return out && rot_dim >= 2 && rot_dim <= kHeadDim && rot_dim % 2 == 0 &&
           (pairs == PKV_ROPE_HALF || pairs == PKV_ROPE_INTERLEAVED);
}

}  // namespace

// A launch's cut, `heads` query rows and `other` bytes of a token besides.  Large
// calls: units of up to four tokens, as many CTAs as the GPU holds with two stages
// of them each.
static RopeTokens tokens_of(const Common &c, int32_t total, int32_t heads, int32_t row_bytes, int32_t other, int nsm, size_t *smem) {
    RopeTokens t;
    std::memset(&t, 0, sizeof(t));
    for (int s = 0; s < c.n_seqs; ++s) t.tok_off[s] = c.seq[s].tok_off;
    t.total = total;
    t.segs = std::max(1, (heads + kSegHeads - 1) / kSegHeads);
    t.bytes = std::min(heads, kSegHeads) * row_bytes + other;
    t.block = 1;
    while (total > 2048 && t.block < kBlockTokens && 2 * t.block * t.bytes <= kStageBytes) t.block *= 2;
    const int64_t units = ((int64_t)(total - 1) / t.block + 1) * t.segs;
    t.units = units <= INT32_MAX / 2 ? static_cast<int32_t>(units) : 0;  // (none: more than a launch takes)
    const int holds = std::min(kCtas, kSmBytes / (2 * t.block * t.bytes + kStaticBytes));
    t.ctas = t.block == 1 ? t.units : std::min(t.units, nsm * std::max(1, holds));
    *smem = static_cast<size_t>(t.ctas < t.units ? 2 : 1) * t.block * t.bytes;
    return t;
}

// A token of 64 query heads, 64 KV heads and an indexer row takes 97 KB; an SM left
// with a small carveout could not take a CTA beside the kernel before.
constexpr int kMaxSmem = std::max((kSegHeads + 2 * 64) * kHeadDim * 2 + kIdxDim * 2, 2 * kStageBytes);
static int set_smem(const void *f) {
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) return PKV_ECUDA;
    return cuda_rc(cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared));
}

int launch_rope_rows(const Common &c, int32_t total_tokens, const pkv_rope &rope, const RopeRows &r, int32_t dim,
                     cudaStream_t stream) {
    int nsm = 0;
    const int rc = sm_count(&nsm);
    if (rc) return rc;
    size_t smem;
    const RopeTokens t = tokens_of(c, total_tokens, c.n_q_heads, dim * 2, 0, nsm, &smem);
    if (t.units == 0) return PKV_EINVAL;
    using Kernel = void (*)(Common, pkv_rope, RopeRows, RopeTokens);
    const Kernel fns[2][3] = {{rope_rows<kIdxDim, kInside>, rope_rows<kIdxDim, kApart>, rope_rows<kIdxDim, kAnyhow>},
                              {rope_rows<kHeadDim, kInside>, rope_rows<kHeadDim, kApart>, rope_rows<kHeadDim, kAnyhow>}};
    static std::atomic<uint64_t> attr_done{0};
    if (once_per_device(attr_done, [&] {
            for (const auto &of_dim : fns)
                for (const Kernel f : of_dim)
                    if (set_smem(reinterpret_cast<const void *>(f)) != PKV_OK) return PKV_ECUDA;
            return PKV_OK;
        }) != PKV_OK)
        return PKV_ECUDA;
    return launch_status(launch_pdl(fns[dim == kHeadDim][mode_of(rope) - kInside], t.ctas, kThreads, smem, stream, c,
                                    rope, r, t));
}

int launch_rope_store(const Common &c, int32_t total_tokens, const pkv_rope *rope, const RopeRows &r, cudaStream_t stream,
                      bool early) {
    int nsm = 0;
    const int rc = sm_count(&nsm);
    if (rc) return rc;
    size_t smem;
    const RopeTokens t = tokens_of(c, total_tokens, rope && r.q ? c.n_q_heads : 0, kHeadDim * 2,
                                   (2 * c.n_kv_heads * kHeadDim + c.idx_dim) * 2, nsm, &smem);
    if (t.units == 0) return PKV_EINVAL;
    pkv_rope none;
    if (!rope) std::memset(&none, 0, sizeof(none));
    using Kernel = void (*)(Common, pkv_rope, RopeRows, RopeTokens, bool);
    const Kernel fns[2][4] = {{rope_store<false, kStill>, rope_store<false, kInside>, rope_store<false, kApart>, rope_store<false, kAnyhow>},
                              {rope_store<true, kStill>, rope_store<true, kInside>, rope_store<true, kApart>, rope_store<true, kAnyhow>}};
    static std::atomic<uint64_t> attr_done{0};
    if (once_per_device(attr_done, [&] {
            for (const auto &of_format : fns)
                for (const Kernel f : of_format)
                    if (set_smem(reinterpret_cast<const void *>(f)) != PKV_OK) return PKV_ECUDA;
            return PKV_OK;
        }) != PKV_OK)
        return PKV_ECUDA;
    return launch_status(launch_pdl(fns[c.kv_fp8 != 0][rope ? mode_of(*rope) : kStill], t.ctas, kThreads, smem, stream,
                                    c, rope ? *rope : none, r, t, early));
}

// ---- entry points -----------------------------------------------------------------

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A row stride of the caller's: 0 stands for packed rows.
static bool row_stride(int64_t given, int64_t packed, int64_t *out) {
    *out = given ? given : packed;
    return *out >= packed && *out % 8 == 0;
}

static bool rope_ok(const pkv_rope *rope, int32_t dim) {
    return rope && rope_shape_ok(rope->rot_dim, rope->pairs, rope) && rope->rot_dim <= dim && std::isfinite(rope->scale) &&
           rope->reserved == 0;
}

static bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

// Rows read and written: apart (rows of other heads between a token's rows, as in
// one projection's output, may interleave), or the same ones in place.
static bool rows_apart(const void *x, int64_t xs, int64_t x_width, const void *out, int64_t os, int64_t out_width, int64_t tokens) {
    const int64_t gap = (static_cast<const char *>(out) - static_cast<const char *>(x)) / 2;
    if (!overlap(x, 2 * ((tokens - 1) * xs + x_width), out, 2 * ((tokens - 1) * os + out_width))) return true;
    if (xs != os || tokens == 1) return false;
    const int64_t m = ((gap % xs) + xs) % xs;  // out's place among x's rows
    return m >= x_width && m + out_width <= xs;
}
static bool in_place_ok(const void *x, int64_t xs, const void *out, int64_t os, int64_t width, int64_t tokens) {
    return x == out ? xs == os : rows_apart(x, xs, width, out, os, width, tokens);
}

}  // namespace pkv

using namespace pkv;

extern "C" int pkv_rope_from_freqs(int32_t rot_dim, int32_t pairs, const double *radians, double scale, pkv_rope *out) {
    if (!rope_shape_ok(rot_dim, pairs, out) || !radians || !std::isfinite(static_cast<float>(scale))) return PKV_EINVAL;
    pkv_rope r;
    std::memset(&r, 0, sizeof(r));
    r.rot_dim = rot_dim;
    r.pairs = pairs;
    r.scale = static_cast<float>(scale);
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!to_turns(radians[i], &r.turns[i])) return PKV_EINVAL;
    *out = r;
    return PKV_OK;
}

extern "C" int pkv_rope_init(int32_t rot_dim, int32_t pairs, double base, int32_t scaling, double factor, int32_t original,
                             double fast, double slow, double scale, pkv_rope *out) {
    if (!rope_shape_ok(rot_dim, pairs, out)) return PKV_EINVAL;
    if (!std::isfinite(base) || !(base > 1.0) || !std::isfinite(scale)) return PKV_EINVAL;
    if (scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_BANDS) return PKV_EINVAL;
    if (scaling != PKV_ROPE_PLAIN && (!std::isfinite(factor) || !(factor >= 1.0))) return PKV_EINVAL;
    const bool parts = scaling == PKV_ROPE_YARN || scaling == PKV_ROPE_BANDS;
    if (parts) {
        if (fast == 0.0) fast = scaling == PKV_ROPE_YARN ? 32.0 : 4.0;
        if (slow == 0.0) slow = 1.0;
        if (original < 1 || !std::isfinite(fast) || !(slow > 0.0) || !(fast > slow)) return PKV_EINVAL;
    }
    if (scaling == PKV_ROPE_NTK && rot_dim < 4) return PKV_EINVAL;
    const double two_pi = 6.283185307179586476925286766559, d = rot_dim;
    if (scaling == PKV_ROPE_NTK) base *= std::pow(factor, d / (d - 2.0));
    if (!std::isfinite(base)) return PKV_EINVAL;
    // the pair that turns n times over the original length: base^(-2i/d) original = 2 pi n
    const auto pair_of = [&](double n) { return d * std::log(original / (two_pi * n)) / (2.0 * std::log(base)); };
    double low = 0.0, high = 0.0;
    if (scaling == PKV_ROPE_YARN) {
        low = std::max(0.0, std::floor(pair_of(fast)));
        high = std::min(d - 1.0, std::ceil(pair_of(slow)));
    }
    double radians[kMaxPairs];
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / d);
        if (scaling == PKV_ROPE_LINEAR) f /= factor;
        if (parts) {
            // how far the pair keeps its frequency, 0 to 1
            const double keep = scaling == PKV_ROPE_YARN ? 1.0 - (i - low) / std::max(high - low, 1e-3)
                                                         : (original * f / two_pi - slow) / (fast - slow);
            const double k = std::min(1.0, std::max(0.0, keep));
            f = f * k + f / factor * (1.0 - k);
        }
        radians[i] = f;
    }
    if (scale == 0.0) scale = scaling == PKV_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return pkv_rope_from_freqs(rot_dim, pairs, radians, scale, out);
}

extern "C" int pkv_rope_rows(const pkv_rope *rope, const pkv_seq *seqs, int32_t n_seqs, const int32_t *pos, int32_t n_heads,
                             int32_t dim, const void *x, int64_t x_stride, void *out, int64_t out_stride,
                             cudaStream_t stream) {
    if ((dim != kHeadDim && dim != kIdxDim) || !rope_ok(rope, dim) || n_heads < 1 || n_heads > 65536) return PKV_EINVAL;
    if (n_seqs < 0 || n_seqs > PKV_MAX_SEQS || (n_seqs > 0 && !seqs)) return PKV_EINVAL;
    Common c;
    std::memset(&c, 0, sizeof(c));
    c.n_seqs = n_seqs;
    c.n_q_heads = n_heads;
    int64_t tokens = 0;
    for (int s = 0; s < n_seqs; ++s) {
        if (seqs[s].len < 0 || seqs[s].n_new < 0 || seqs[s].n_new > seqs[s].len) return PKV_EINVAL;
        c.seq[s].len = seqs[s].len;
        c.seq[s].n_new = seqs[s].n_new;
        c.seq[s].tok_off = static_cast<int32_t>(tokens);
        tokens += seqs[s].n_new;
        if (tokens > INT32_MAX / 2) return PKV_EINVAL;
    }
    RopeRows r;
    std::memset(&r, 0, sizeof(r));
    const int64_t width = (int64_t)n_heads * dim;
    if (!row_stride(x_stride, width, &r.q_stride) || !row_stride(out_stride, width, &r.q_out_stride)) return PKV_EINVAL;
    if (tokens == 0) return PKV_OK;
    if (!x || !out || !aligned16(x) || !aligned16(out) || !in_place_ok(x, r.q_stride, out, r.q_out_stride, width, tokens))
        return PKV_EINVAL;
    r.q = static_cast<const uint16_t *>(x);
    r.q_out = static_cast<uint16_t *>(out);
    r.pos = pos;
    return launch_rope_rows(c, static_cast<int32_t>(tokens), *rope, r, dim, stream);
}

extern "C" int pkv_rope_store(const pkv_layout *L, const pkv_seq *seqs, int32_t n_seqs, int32_t layer, const pkv_rope *rope,
                              const int32_t *pos, int32_t n_q_heads, const void *q, int64_t q_stride, void *q_out,
                              int64_t q_out_stride, const void *k_new, int64_t k_stride, const void *v_new,
                              int64_t v_stride, const void *ik_new, int64_t ik_stride, int32_t *dev_status,
                              cudaStream_t stream) {
    Common c;
    int rc = fill_common(L, seqs, n_seqs, layer, L ? L->n_kv_heads : 1, dev_status, &c);
    if (rc) return rc;
    if (!rope_ok(rope, kHeadDim)) return PKV_EINVAL;
    int64_t tokens = 0;
    for (int s = 0; s < c.n_seqs; ++s) tokens += c.seq[s].n_new;
    RopeRows r;
    std::memset(&r, 0, sizeof(r));
    const int64_t kv = (int64_t)L->n_kv_heads * kHeadDim;
    if (!row_stride(k_stride, kv, &r.k_stride) || !row_stride(v_stride, kv, &r.v_stride)) return PKV_EINVAL;
    if (L->idx_dim && !row_stride(ik_stride, L->idx_dim, &r.ik_stride)) return PKV_EINVAL;
    if (q) {
        if (n_q_heads < 1 || n_q_heads > 65536) return PKV_EINVAL;
        const int64_t width = (int64_t)n_q_heads * kHeadDim;
        if (!row_stride(q_stride, width, &r.q_stride) || !row_stride(q_out_stride, width, &r.q_out_stride)) return PKV_EINVAL;
        if (tokens > 0 && (!q_out || !aligned16(q) || !aligned16(q_out) ||
                           !in_place_ok(q, r.q_stride, q_out, r.q_out_stride, width, tokens)))
            return PKV_EINVAL;
        c.n_q_heads = n_q_heads;
    }
    if (tokens == 0) return PKV_OK;
    if (!k_new || !v_new || (L->idx_dim && !ik_new)) return PKV_EINVAL;
    if (!aligned16(k_new) || !aligned16(v_new) || (L->idx_dim && !aligned16(ik_new))) return PKV_EINVAL;
    // a token's queries are written while other tokens' keys and values are still read
    if (q) {
        const int64_t width = (int64_t)n_q_heads * kHeadDim;
        if (!rows_apart(k_new, r.k_stride, kv, q_out, r.q_out_stride, width, tokens) ||
            !rows_apart(v_new, r.v_stride, kv, q_out, r.q_out_stride, width, tokens) ||
            (L->idx_dim && !rows_apart(ik_new, r.ik_stride, L->idx_dim, q_out, r.q_out_stride, width, tokens)))
            return PKV_EINVAL;
    }
    r.q = static_cast<const uint16_t *>(q);
    r.q_out = static_cast<uint16_t *>(q_out);
    r.k = static_cast<const uint16_t *>(k_new);
    r.v = static_cast<const uint16_t *>(v_new);
    r.ik = static_cast<const uint16_t *>(ik_new);
    r.pos = pos;
    return launch_rope_store(c, static_cast<int32_t>(tokens), rope, r, stream, false);
}
