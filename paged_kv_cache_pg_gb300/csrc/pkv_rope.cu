// Rotary positions: rows rotated by their tokens' positions, alone
// (pkv_rope_rows) or on the way into the pages (pkv_rope_store).
//
// Pair i of a row at position p turns by p f_i.  The frequencies come as
// fractions of a turn times 2^64, so p times one, modulo 2^64, is the angle
// without its whole turns, exact to 2^-64 of a turn a position; its top 32 bits
// (a signed fraction of a half turn) go to sincospif.  In float32 radians a
// position of 10^6 would leave 0.03 of the fastest pair's angle to chance.
//
// A CTA takes one token, or four of large calls, and computes each token's
// cosines and sines once, into shared memory, for all of its heads (16 query
// rows and 2 key rows use the same 32 to 128 pairs); with positions from the
// launch parameters that happens before the grid-dependency wait.  A warp then
// takes a row of 256 elements (two rows of 128), a lane 16 bytes of it; the
// other elements of a lane's pairs (PKV_ROPE_HALF) are a second 16-byte load of
// the row, which L1 has, or eight scalar ones where half of rot_dim is not a
// multiple of 8.  Values and indexer rows are copied by the same warps.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pkv_dev.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kBlockTokens = 4;  // of a CTA of large calls

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

// Elements 8 ch .. 8 ch + 7 of `row`, rotated, as float32.  cs: the token's
// (cosine, sine) pairs.  Plain loads: the row may be rotated in place.
__device__ __forceinline__ void rotated(const uint16_t *row, int ch, int rot, int interleaved, const float2 *cs,
                                        float (&x)[8]) {
    widen(*(reinterpret_cast<const uint4 *>(row) + ch), x);
    const int e0 = 8 * ch, half = rot >> 1;
    if (e0 >= rot) return;
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            if (e0 + e < rot) {
                const float2 t = cs[(e0 + e) >> 1];
                const float a = x[e], b = x[e + 1];
                x[e] = a * t.x - b * t.y;
                x[e + 1] = b * t.x + a * t.y;
            }
    } else if ((half & 7) == 0) {
        const bool first = e0 < half;
        float y[8];
        widen(*(reinterpret_cast<const uint4 *>(row) + (first ? ch + (half >> 3) : ch - (half >> 3))), y);
        const float2 *const t = cs + (first ? e0 : e0 - half);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * t[e].x + (first ? -y[e] : y[e]) * t[e].y;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = e0 + e;
            if (i >= rot) continue;
            const bool first = i < half;
            const float y = __uint_as_float(static_cast<uint32_t>(row[first ? i + half : i - half]) << 16);
            const float2 t = cs[first ? i : i - half];
            x[e] = x[e] * t.x + (first ? -y : y) * t.y;
        }
    }
}

// The tables of a CTA's tokens.
__device__ __forceinline__ void fill_turns(const Common &c, const pkv_rope &rope, const int32_t *pos, int32_t tok0, int n,
                                           float2 *cs) {
    const int pairs = rope.rot_dim >> 1;
    for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
        const int k = i / pairs, j = i - k * pairs, tok = tok0 + k;
        int32_t p;
        if (pos) {
            p = __ldg(pos + tok);
        } else {
            const int s = find_seq(c.n_seqs, tok, [&](int t) { return c.seq[t].tok_off; });
            p = c.seq[s].len - c.seq[s].n_new + (tok - c.seq[s].tok_off);
        }
        cs[k * kMaxPairs + j] = turn(rope.turns[j], p, rope.scale);
    }
    __syncthreads();
}

// Rows of kDim elements, c.n_q_heads a token, per CTA `block` tokens.
template <int kDim>
__global__ void __launch_bounds__(kThreads)
    rope_rows(const __grid_constant__ Common c, const __grid_constant__ pkv_rope rope, const __grid_constant__ RopeRows r,
              int32_t total_tokens, int32_t block) {
    __shared__ float2 cs[kBlockTokens * kMaxPairs];
    constexpr int kChunks = kDim / 8, kRowsWarp = 32 / kChunks;
    const int32_t tok0 = blockIdx.x * block;
    const int n = min(block, total_tokens - tok0);
    if (r.pos) pdl_wait();
    fill_turns(c, rope, r.pos, tok0, n, cs);
    if (!r.pos) pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();  // nothing here is read before a grid-dependency wait
    const int lane = threadIdx.x & 31, ch = lane % kChunks, sub = lane / kChunks;
    const int rows = n * c.n_q_heads;
    for (int i = (threadIdx.x >> 5) * kRowsWarp; i < rows; i += kWarps * kRowsWarp) {
        const int at = i + sub, k = at / c.n_q_heads, h = at - k * c.n_q_heads;
        float x[8];
        if (at < rows)
            rotated(r.q + (tok0 + k) * r.q_stride + h * kDim, ch, rope.rot_dim, rope.pairs, cs + k * kMaxPairs, x);
        __syncwarp();  // every lane of the row has read what it turns, which may be in place
        if (at < rows)
            *(reinterpret_cast<uint4 *>(r.q_out + (tok0 + k) * r.q_out_stride + h * kDim) + ch) = narrow(x);
    }
}

// A token's rows: its queries (when given), keys, values, indexer row.
template <bool kFp8>
__global__ void __launch_bounds__(kThreads)
    rope_store(const __grid_constant__ Common c, const __grid_constant__ pkv_rope rope, const __grid_constant__ RopeRows r,
               int32_t total_tokens, int32_t block) {
    __shared__ float2 cs[kBlockTokens * kMaxPairs];
    const int32_t tok0 = blockIdx.x * block;
    const int n = min(block, total_tokens - tok0);
    const int H = c.n_kv_heads, nq = r.q ? c.n_q_heads : 0;
    const int per = nq + 2 * H + (c.idx_dim ? 1 : 0);
    if (r.pos) pdl_wait();
    fill_turns(c, rope, r.pos, tok0, n, cs);
    if (!r.pos) pdl_wait();
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < n * per; i += kWarps) {
        const int k = i / per;
        int row = i - k * per;
        const int64_t tok = tok0 + k;
        const float2 *const t = cs + k * kMaxPairs;
        float x[8];
        if (row < nq) {
            rotated(r.q + tok * r.q_stride + row * kHeadDim, lane, rope.rot_dim, rope.pairs, t, x);
            __syncwarp();  // as in rope_rows
            *(reinterpret_cast<uint4 *>(r.q_out + tok * r.q_out_stride + row * kHeadDim) + lane) = narrow(x);
            continue;
        }
        row -= nq;
        const int s = find_seq(c.n_seqs, tok0 + k, [&](int t) { return c.seq[t].tok_off; });
        const SeqDev &sd = c.seq[s];
        // every lane reads the table's entry (one address); one reports it
        int32_t in_page;
        int64_t page = 0;
        const int32_t place = sd.len - sd.n_new + (tok0 + k - sd.tok_off);
        if (sd.table) {
            const int32_t p = place / sd.ptok;
            in_page = place - p * sd.ptok;
            const int32_t id = __ldg(sd.table + p);
            if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(sd.n_pages)) {
                if (lane == 0 && c.status) atomicOr(c.status, PKV_DEV_BAD_PAGE);
                continue;
            }
            page = (int64_t)id * sd.ps;
        } else {
            in_page = place;
        }
        uint16_t *const base = const_cast<uint16_t *>(sd.layer_base) + page;
        if (row < 2 * H) {
            const bool v = row >= H;
            const int head = v ? row - H : row;
            if (v) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(r.v + tok * r.v_stride + head * kHeadDim) + lane);
                if constexpr (!kFp8) {
                    *(reinterpret_cast<uint4 *>(base + off_v(H, sd.ptok, head, in_page)) + lane) = u;
                    continue;
                }
                widen(u, x);
            } else {
                rotated(r.k + tok * r.k_stride + head * kHeadDim, lane, rope.rot_dim, rope.pairs, t, x);
            }
            if constexpr (kFp8) {
                uint8_t *const b8 = reinterpret_cast<uint8_t *>(base);
                uint2 codes;
                const float scale = quantize_row8f(x, &codes);
                *reinterpret_cast<uint2 *>(b8 + off8_code(v, H, sd.ptok, head, in_page) + lane * 8) = codes;
                if (lane == 0) *reinterpret_cast<float *>(b8 + off8_scale(v, H, sd.ptok, head, in_page)) = scale;
            } else {
                *(reinterpret_cast<uint4 *>(base + off_k(sd.ptok, head, in_page)) + lane) = narrow(x);
            }
        } else if (lane < kIdxDim / 8) {
            *(reinterpret_cast<uint4 *>(base + off_ik_f(kFp8, H, c.idx_dim, sd.ptok, in_page)) + lane) =
                __ldg(reinterpret_cast<const uint4 *>(r.ik + tok * r.ik_stride) + lane);
        }
    }
    pdl_trigger_after_writes();  // the next decode may read these rows early
}

// Tokens a CTA: one while the CTAs of one token each fit the GPU about twice
// over, else four.
int block_of(int32_t tokens) { return tokens > 2048 ? kBlockTokens : 1; }

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

int launch_rope_rows(const Common &c, int32_t total_tokens, const pkv_rope &rope, const RopeRows &r, int32_t dim,
                     cudaStream_t stream) {
    const int block = block_of(total_tokens);
    return launch_status(launch_pdl(dim == kHeadDim ? rope_rows<kHeadDim> : rope_rows<kIdxDim>,
                                    static_cast<unsigned>((total_tokens - 1) / block + 1), kThreads, 0, stream, c, rope,
                                    r, total_tokens, block));
}

int launch_rope_store(const Common &c, int32_t total_tokens, const pkv_rope &rope, const RopeRows &r,
                      cudaStream_t stream) {
    const int block = block_of(total_tokens);
    return launch_status(launch_pdl(c.kv_fp8 ? rope_store<true> : rope_store<false>,
                                    static_cast<unsigned>((total_tokens - 1) / block + 1), kThreads, 0, stream, c, rope,
                                    r, total_tokens, block));
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

// Rows read and written: the same ones in place, or apart (rows of other heads
// between a token's rows, as in one projection's output, may interleave).
static bool in_place_ok(const void *x, int64_t xs, const void *out, int64_t os, int64_t width, int64_t tokens) {
    if (x == out) return xs == os;
    const int64_t gap = (static_cast<const char *>(out) - static_cast<const char *>(x)) / 2;
    if (!overlap(x, 2 * ((tokens - 1) * xs + width), out, 2 * ((tokens - 1) * os + width))) return true;
    if (xs != os) return false;
    const int64_t m = ((gap % xs) + xs) % xs;  // out's place among x's rows
    return m >= width && m + width <= xs;
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
    r.q = static_cast<const uint16_t *>(q);
    r.q_out = static_cast<uint16_t *>(q_out);
    r.k = static_cast<const uint16_t *>(k_new);
    r.v = static_cast<const uint16_t *>(v_new);
    r.ik = static_cast<const uint16_t *>(ik_new);
    r.pos = pos;
    return launch_rope_store(c, static_cast<int32_t>(tokens), *rope, r, stream);
}
