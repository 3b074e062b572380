// Shared by the kernels that read a paged cache for single tokens: the work's cut into pieces, the
// producer warp with its ring of tiles, the records of pieces and their join.
#pragma once

#include <cuda.h>

#include "lola_attn.cuh"
#include "lola_tc.cuh"

namespace lola {
namespace {

using namespace tc;

__device__ int32_t g_status;

constexpr int kTile = 64;                 // tokens per tile
constexpr int kCons = 256;                // consumer threads
constexpr int kThreads = kCons + kWarp;
constexpr int kPieces = 152;              // one CTA per SM
constexpr int kRows = 16;                 // query rows of a row group (at most)
constexpr int kJoin = 16;                 // pieces joined at a time
constexpr float kRaise = 8.0f;            // bf16: m is set this far above a maximum (log2), and raised when one passes it
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 50000000ull;   // ... for copies in flight, when a wait has given up

struct Maps {
    CUtensorMap k, v;   // [n_pages * Hkv][page][d] as 128-byte columns, boxes of min(page, a tile's tokens) rows (e4m3: of 128
                        // bytes, which are two tokens at d = 64)
};

struct Args {
    PagedArgs p;        // SH: of the prefixes, or of the sequences
    PagedArgs pre;      // PRE: the prefixes
    Sharing sh;         // SH, PRE: whose rows see them
    Parts parts;        // SH: what is left of them
    Rows Q, O;
    float* lse;
    float* part;        // workspace: records, then the joins' cells
    uint64_t tag;       // this call's mark in the cells (the low 8 bits are 0)
    float scale_log2;
    int give_up;        // lola_selftest_attn_wait: a tile at which every third CTA gives up
    int RG, I;          // row groups per key/value head; items (row groups) per sequence
};

// T: the cache's numbers (uint8_t: e4m3, whose powers of two, a byte a token, follow the ring; a tile has twice the
// tokens, as the producers take some 600 clocks for one, whatever its bytes)
template <typename T, int D> struct Cfg {
    static constexpr int kTokens = sizeof(T) == 1 ? 128 : kTile;   // of a tile
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kHalf = kTokens * kRowBytes;              // K or V of a tile
    static constexpr int kScales = sizeof(T) == 1 ? 2 * kTokens : 0;   // bytes of powers of a tile
    static constexpr int kFull = sizeof(T) == 1 ? 1 + kWarp : 1;   // arrivals that a loaded tile takes
    static constexpr int kMost = 12;
    static constexpr int kStages = 196608 / (2 * kHalf + kScales) > kMost ? kMost : 196608 / (2 * kHalf + kScales);
    static constexpr int kSmem = kStages * (2 * kHalf + kScales) + 1024;
};
// ... with a ring of S stages
template <typename B, int S> struct Ring : B {
    static constexpr int kStages = S, kSmem = S * (2 * B::kHalf + B::kScales) + 1024;
};

// ---- the workspace: per piece four records of (O [16][d], m [16], l [16]) -- its first segment's (slot
// 0), its last one's (1), and the joins of up to 16 pieces that begin with one of them (2, 3) -- and as
// many cells that count a join's arrivals ----
constexpr int kSlots = 4;
__host__ __device__ constexpr int64_t record_floats(int d) { return kRows * (int64_t)d + 2 * kRows; }
template <int D>
__device__ __forceinline__ float* record(const Args& a, int piece, int slot) {
    return a.part + ((int64_t)piece * kSlots + slot) * record_floats(D);
}
template <int D>
__device__ __forceinline__ unsigned long long* cell(const Args& a, int piece, int slot) {
    return reinterpret_cast<unsigned long long*>(a.part + (int64_t)kPieces * kSlots * record_floats(D)) + piece * kSlots + slot;
}

// ---- query rows: G of a sequence, or (SH) those of all sequences that share a prefix, sequence by sequence.  SH: the
// segments' parts are left for another kernel, none of them is joined here ----
struct Group {
    int m0, rows;          // first sequence
    int RG, I;             // row groups per key/value head; items
};
template <bool SH, int ROWS = kRows> __device__ __forceinline__ Group group_of(const Args& a, int b, int* bits = nullptr) {
    Group g;
    if constexpr (SH) {
        int n = a.sh.each ? 1 : a.sh.n_seq, bad = 0;
        g.m0 = a.sh.each ? b : 0;
        if (a.sh.cu) seq_rows(a.sh.cu, b, a.sh.n_seq, &g.m0, &n, &bad);
        if (bits) *bits |= bad;
        g.rows = n * a.p.G;
        g.RG = (g.rows + ROWS - 1) / ROWS;
        g.I = a.p.Hkv * g.RG;
    } else {
        g.m0 = b;
        g.rows = a.p.G;
        g.RG = a.RG;
        g.I = a.I;
    }
    return g;
}

// Tiles of sequence b, for each of its items: at least one, so that an empty sequence's output
// is written too.
template <int TILE = kTile>
__device__ __forceinline__ int tiles_of(int64_t tokens) { return tokens <= 0 ? 1 : (int)((tokens + TILE - 1) / TILE); }

// ---- PRE: the tiles of a sequence are those of its prefix, then its own ----
struct View {
    int g, tokens, tiles;      // the prefix (-1: none), its tokens and tiles
};
template <int TILE> __device__ __forceinline__ View view_of(const Args& a, int b, int* bits) {
    View v{-1, 0, 0};
    for (int x = 0; x < a.pre.n_seq; ++x) {
        int lo = 0, n = a.p.n_seq;
        if (a.sh.cu) seq_rows(a.sh.cu, x, a.p.n_seq, &lo, &n, bits);
        if (b >= lo && b < lo + n) v.g = x;
    }
    if (v.g >= 0) v.tokens = (int)paged_tokens(a.pre, a.pre.kv_len[v.g]);
    v.tiles = (v.tokens + TILE - 1) / TILE;
    return v;
}
// tiles of sequence b, which has so many tokens of its own
template <int TILE, bool PRE> __device__ __forceinline__ int item_tiles(const Args& a, int b, int64_t tokens, int* bits) {
    if constexpr (!PRE) return tiles_of<TILE>(tokens);
    const int pre = view_of<TILE>(a, b, bits).tiles;
    return pre + (pre > 0 && tokens <= 0 ? 0 : tiles_of<TILE>(tokens));
}

// Units of sequence (or prefix) b: a prefix without tokens or sequences has none.
template <bool SH, int TILE = kTile, int ROWS = kRows, bool PRE = false>
__device__ __forceinline__ int64_t units_of(const Args& a, int b, int* bits) {
    if constexpr (PRE) return (int64_t)item_tiles<TILE, true>(a, b, paged_tokens(a.p, a.p.kv_len[b]), bits) * a.I;
    const int64_t tokens = paged_tokens(a.p, a.p.kv_len[b]);
    if (SH && tokens == 0) return 0;
    return (int64_t)tiles_of<TILE>(tokens) * group_of<SH, ROWS>(a, b, bits).I;
}

// Pieces of `total` units: none is empty.
__device__ __forceinline__ int pieces_of(int64_t total) { return (int)min((int64_t)kPieces, total); }

// One segment of the piece, published by the producer: `R` < 0 ends the consumers.
struct Seg {
    int b, h0, R;          // (first) sequence, first query head, query rows
    int r0;                // SH: the first row's number among the prefix' rows of this key head
    int tiles, n0;         // tiles of the segment, number of its first one in the ring's order
    int len;               // tokens of the sequence from the segment's first tile on
    int whole;             // it covers the whole item
    int k, np, c0, s0;     // else: piece k of np, the first of them c0, whose record is slot s0
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store4(float* o, const float (&y)[4]) {
    *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* o, const float (&y)[4]) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
}

__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, int* abort_sm) {
    uint64_t start = 0;
    for (int it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*reinterpret_cast<volatile int*>(abort_sm)) return false;
        const uint64_t now = globaltimer_ns();
        if (it == 0) start = now;
        else if (now - start > kWaitNs) {
            *abort_sm = 1;
            return false;
        }
    }
}
// 4 bytes, asynchronously
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// the producer has armed tile n's stage: only then does the parity of n's phase tell it from the one
// before (a group that has not waited for that one, which was another group's, would pass at once)
__device__ __forceinline__ bool issued_wait(const int* issued, int n, int* abort_sm) {
    if (*reinterpret_cast<const volatile int*>(issued) > n) return true;
    const uint64_t start = globaltimer_ns();
    while (*reinterpret_cast<const volatile int*>(issued) <= n) {
        if (*reinterpret_cast<volatile int*>(abort_sm)) return false;
        if (globaltimer_ns() - start > kWaitNs) {
            *abort_sm = 1;
            return false;
        }
    }
    return true;
}
// *count has come to `want`
__device__ __forceinline__ bool count_wait(const int* count, int want, int* abort_sm) {
    const uint64_t start = globaltimer_ns();
    while (*reinterpret_cast<const volatile int*>(count) < want) {
        if (*reinterpret_cast<volatile int*>(abort_sm)) return false;
        if (globaltimer_ns() - start > kWaitNs) {
            *abort_sm = 1;
            return false;
        }
    }
    return true;
}
// barrier `id` of a group of NT threads that also tells all of them whether one had x (so that a
// wait that gave up ends the whole group, and no barrier is left waiting)
template <int NT>
__device__ __forceinline__ bool group_or(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "n"(NT)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Barriers: a ring stage is full / empty; a segment slot (descriptor and Q rows) is full / empty.
template <int S, int NS = 2> struct Bars {
    uint64_t full[S], empty[S], seg_full[NS], seg_empty[NS];
    int issued;      // tiles whose stage is armed
    int ahead;       // tiles whose V codes' copies are on their way (e4m3: by a warp of their own, which may be ahead)
    int given;       // segment slots given to the consumers, when the producer is done
    int arrived[2];  // this piece's record of that slot has been counted
};

// Which piece this CTA is and where it begins (all threads): false if there is none.
struct Start {
    int64_t total, u0, u1, rem;   // units; rem: the first unit's number inside its sequence
    int N, b;                     // pieces; the first unit's sequence
    int piece;
};
template <bool SH, int NT = kThreads, int TILE = kTile, int ROWS = kRows, bool PRE = false>
__device__ __forceinline__ bool find_start(const Args& a, Start* st) {
    const PagedArgs& p = a.p;
    __shared__ int64_t sums[NT / kWarp];
    __shared__ int found_b;
    __shared__ int64_t found_r;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    int bits = 0;
    auto count = [&](int b) -> int64_t { return b < p.n_seq ? units_of<SH, TILE, ROWS, PRE>(a, b, &bits) : 0; };
    const int64_t own = count(threadIdx.x);            // (the whole of it up to NT sequences)
    int64_t rest = 0;
    for (int b = threadIdx.x + NT; b < p.n_seq; b += NT) rest += count(b);
    st->total = block_total<NT>(own + rest, sums);
    st->N = pieces_of(st->total);
    st->piece = (int)blockIdx.x;
    if ((SH || PRE) && bits) atomicOr(&g_status, bits);
    if ((int)blockIdx.x >= st->N) return false;
    st->u0 = split_at(st->total, st->N, blockIdx.x);
    st->u1 = split_at(st->total, st->N, blockIdx.x + 1);
    int64_t before = 0;
    for (int base = 0; base < p.n_seq; base += NT) {
        const int64_t x = base == 0 ? own : count(base + threadIdx.x);
        int64_t inc = x;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == kWarp - 1) sums[warp] = inc;
        __syncthreads();
        int64_t pre = before, all = before;
#pragma unroll
        for (int w = 0; w < NT / kWarp; ++w) {
            if (w < warp) pre += sums[w];
            all += sums[w];
        }
        const int64_t lo = pre + inc - x;
        if (st->u0 >= lo && st->u0 < lo + x) {
            found_b = base + threadIdx.x;
            found_r = st->u0 - lo;
        }
        if (st->u0 < all) break;
        before = all;
    }
    __syncthreads();
    st->b = found_b;
    st->rem = found_r;
    return true;
}

// The segment [t0, t1) of an item of `tiles` tiles as one piece of it: the item's first unit is xs.
__device__ __forceinline__ void place_piece(const Start& st, int64_t xs, int tiles, Seg* g) {
    g->c0 = split_of(st.total, st.N, xs);
    g->np = split_of(st.total, st.N, xs + tiles - 1) - g->c0 + 1;
    g->k = st.piece - g->c0;
    g->s0 = xs != split_at(st.total, st.N, g->c0);
}

// The producer warp: segments and their tiles, in order.  A tile's pages outside the cache are not
// loaded; bit x of bad_sm marks the tile's x-th token box.  Segment i goes to slot i % NS.
// TQ: the queries' numbers.  e4m3: three warps (`part` 0-2: codes of K, of V, powers of both) that walk the segments side
// by side, as each copy takes its thread some 180 clocks to issue, and a tile of codes half a tile's time at most (all
// copies by one warp: 64 sequences of 1000-8000 tokens, 32/8 heads, d = 128, 117 us).  The first of them does the rest.
// The powers come four bytes a lane, past the tensor unit, whose small copies take as long as its large ones.
template <typename T, typename TQ, int D, int NS, bool SH, typename C = Cfg<T, D>, int ROWS = kRows, bool PRE = false, typename B>
__device__ __forceinline__ void produce(const Maps& maps, const Args& a, const Start& st, uint32_t ring, uint32_t qs,
                                        uint32_t q_pitch, B& bars, Seg* segs, uint32_t* bad_sm, int* abort_sm, int lane, int part = 0) {
    constexpr bool kParts = C::kScales > 0;
    const bool first = !kParts || part == 0;
    const PagedArgs& p = a.p;
    constexpr uint32_t kQBytes = D * (uint32_t)sizeof(TQ);
    const int box = min(p.page, C::kTokens), lb = 31 - __clz(box), nbox = C::kTokens >> lb;   // tokens of a box, boxes of a tile
    int b = st.b;
    Group gr = group_of<SH>(a, b);
    int lens_b = b;                                               // the lanes hold 32 sequences' lengths
    int lens = b + lane < p.n_seq ? p.kv_len[b + lane] : 0;
    int64_t tokens = paged_tokens(p, __shfl_sync(0xffffffffu, lens, 0));
    int ignored = 0;
    [[maybe_unused]] View view{-1, 0, 0};
    if constexpr (PRE) view = view_of<C::kTokens>(a, b, &ignored);
    int tiles = item_tiles<C::kTokens, PRE>(a, b, tokens, &ignored), t0, item = divide(st.rem, tiles, &t0);
    int64_t u = st.u0;
    int n = 0, i = 0, held_b = -1, held = -1;
    int held_c = 0;                                           // ... and 32 page-table columns of held_b
    bool ok = true;
    while (u < st.u1 && ok) {
        const int t1 = (int)min((int64_t)tiles, t0 + (st.u1 - u));
        const int hk = item / gr.RG, r0 = (item % gr.RG) * kRows, h0 = hk * p.G + (SH ? 0 : r0), R = min(kRows, gr.rows - r0);
        // ---- the segment's descriptor and Q rows ----
        const int slot = i % NS;
        if (first && i >= NS) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.seg_empty[slot]), (uint32_t)(i / NS - 1) & 1, abort_sm));
        if (!ok) break;
        if (first && lane == 0) {
            Seg g;
            g.b = gr.m0;
            g.h0 = h0;
            g.r0 = SH ? r0 : 0;
            g.R = R;
            g.tiles = t1 - t0;
            g.n0 = n;
            g.len = (int)max((int64_t)0, tokens - (int64_t)t0 * C::kTokens);
            g.whole = t0 == 0 && t1 == tiles;
            g.k = g.np = g.c0 = g.s0 = 0;
            if (!g.whole) place_piece(st, u - t0, tiles, &g);
            segs[slot] = g;
            if (p.kv_len[b] > tokens && tokens > 0) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
            if (PRE && view.g >= 0 && a.pre.kv_len[view.g] > view.tokens) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
            mbar_expect(smem_u32(&bars.seg_full[slot]), (uint32_t)R * kQBytes);
        }
        __syncwarp();
        if (first && lane < R) {
            const int seq = SH ? gr.m0 + (r0 + lane) / p.G : b, h = SH ? h0 + (r0 + lane) % p.G : h0 + lane;
            bulk_load(qs + (uint32_t)slot * ROWS * q_pitch + lane * q_pitch,
                      a.Q.data + ((int64_t)seq * a.Q.row + (int64_t)h * a.Q.head) * (int)sizeof(TQ), kQBytes, smem_u32(&bars.seg_full[slot]));
        }
        ++i;
        // ---- its tiles ----
        const bool give_up = gives_up(a.give_up, n, t1 - t0);
        const int stop = give_up ? t0 + a.give_up - n : t1;
        for (int t = t0; t < stop; ++t, ++n) {
            const int s = n % C::kStages;
            if (n >= C::kStages) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.empty[s]), (uint32_t)(n / C::kStages - 1) & 1, abort_sm));
            if (!ok) break;
            // (positions fit 31 bits, but for the boxes behind the last token's)
            const bool pre = PRE && t < view.tiles;
            const uint32_t pos = (uint32_t)(PRE && !pre ? t - view.tiles : t) * C::kTokens, have = (uint32_t)(pre ? view.tokens : tokens);
            const int entry = PRE ? 2 * b + pre : b;              // (whose columns are held)
            const int col = (int)(pos >> p.page_log2);
            const int used = have > pos ? min(nbox, (int)((have - pos + box - 1) >> lb)) : 0;     // boxes with tokens
            if (held_b != entry || col < held_c || col + used > held_c + 32) {
                held_b = entry;
                held_c = col;
                const int64_t c = (int64_t)(col + lane) << p.page_log2;
                held = c >= (int64_t)have ? 0 : pre ? paged_page(a.pre, view.g, c) : paged_page(p, b, c);
            }
            // lanes 0 .. used - 1: a box of K each; lanes 16 ..: of V (e4m3: this warp's part)
            const int x = lane & 15;
            const int page = __shfl_sync(0xffffffffu, held, ((int)((pos + x * box) >> p.page_log2) - held_c) & 31);
            const bool mine = x < used, bad = mine && page < 0;
            const uint32_t bad_mask = __ballot_sync(0xffffffffu, bad) & 0xffffu;
            if (first && lane == 0) {
                if (bad_mask) atomicOr(&g_status, (int)LOLA_ATTN_BAD_PAGE);
                bad_sm[s] = PRE ? bad_mask | (have > pos ? min(have - pos, (uint32_t)C::kTokens) : 0u) << 16 : bad_mask;
                mbar_expect(smem_u32(&bars.full[s]), (uint32_t)(2 * (used - __popc(bad_mask)) * box * C::kRowBytes));
                *reinterpret_cast<volatile int*>(&bars.issued) = n + 1;
            }
            if (kParts && part == 1 && lane == 0) *reinterpret_cast<volatile int*>(&bars.ahead) = n + 1;
            __syncwarp();
            if constexpr (kParts) {
                if (part == 2) {
                    const int k = 4 * lane, of = __shfl_sync(0xffffffffu, held, ((int)((pos + k) >> p.page_log2) - held_c) & 31);
                    if ((k >> lb) < used && of >= 0) {
                        const int64_t at = ((int64_t)of * p.Hkv + hk) * p.page + ((pos + k) & (p.page - 1));
                        const uint32_t to = ring + (uint32_t)C::kStages * 2 * C::kHalf + (uint32_t)s * C::kScales + k;
                        cp_async4(to, p.Ks + at);
                        cp_async4(to + C::kTokens, p.Vs + at);
                    }
                    cp_async_arrive_noinc(smem_u32(&bars.full[s]));
                    continue;
                }
            }
            if (mine && !bad && (!kParts || lane < 16)) {
                const int at = (int)((pos + x * box) & (p.page - 1)), v = kParts ? part : lane >> 4;
                tma_load4(ring + (uint32_t)s * 2 * C::kHalf + v * C::kHalf + x * (uint32_t)(box * C::kRowBytes), v ? &maps.v : &maps.k, 0,
                          kParts ? at * D / 128 : at, 0, page * p.Hkv + hk, smem_u32(&bars.full[s]));
            }
        }
        if (give_up) {
            if (first && lane == 0) *reinterpret_cast<volatile int*>(abort_sm) = 1;
            ok = false;
        }
        u += t1 - t0;
        t0 = 0;
        if (++item == gr.I && u < st.u1) {
            item = 0;
            do {
                ++b;
                if (b >= lens_b + 32) {
                    lens_b = b;
                    lens = b + lane < p.n_seq ? p.kv_len[b + lane] : 0;
                }
                tokens = paged_tokens(p, __shfl_sync(0xffffffffu, lens, b - lens_b));
                gr = group_of<SH>(a, b);
            } while (SH && (tokens == 0 || gr.I == 0));               // (units are left: there is such a prefix)
            if constexpr (PRE) view = view_of<C::kTokens>(a, b, &ignored);
            tiles = item_tiles<C::kTokens, PRE>(a, b, tokens, &ignored);
        }
    }
    if (!first) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    // the consumers' end
    for (int e = 0; e < NS && ok; ++e, ++i) {
        const int slot = i % NS;
        if (i >= NS) ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&bars.seg_empty[slot]), (uint32_t)(i / NS - 1) & 1, abort_sm));
        if (ok && lane == 0) {
            segs[slot].R = -1;
            mbar_arrive1(smem_u32(&bars.seg_full[slot]));
        }
    }
    if (lane == 0) {
        if (!ok) atomicOr(&g_status, (int)LOLA_ATTN_TIMEOUT);
        bars.given = i;
    }
}

// Whether sequence b has a token that can be seen (on a page of the cache).
__device__ __forceinline__ bool sees_token(const PagedArgs& p, int b) {
    const int64_t tokens = paged_tokens(p, p.kv_len[b]);
    for (int64_t pos = 0; pos < tokens; pos += p.page)
        if (paged_page(p, b, pos) >= 0) return true;
    return false;
}

// ... or its prefix has
__device__ __forceinline__ bool sees_any(const Args& a, int b) {
    if (sees_token(a.p, b)) return true;
    int ignored = 0;
    const int g = a.pre.n_seq > 0 ? view_of<kTile>(a, b, &ignored).g : -1;
    return g >= 0 && sees_token(a.pre, g);
}

// Where a segment that is a piece of its item leaves its part.
template <int D, bool SH> __device__ __forceinline__ float* segment_record(const Args& a, const Seg& g) {
    const int slot = g.k == 0 ? g.s0 : 0;
    if constexpr (SH) return a.parts.rec + ((int64_t)blockIdx.x * 2 + slot) * part_record(kRows, D);
    else return record<D>(a, blockIdx.x, slot);
}

// One row's 4 columns c .. c + 3: o, when all of the item's tokens are in, or a record.  SH: left for the
// kernel that joins them.
template <typename T, int D, bool SH>
__device__ __forceinline__ void write_out(const Args& a, const Seg& g, bool whole, float* rec, int r, int c, float (&y)[4], float M, float L) {
    if constexpr (SH) {
        const Parts& q = a.parts;
        const int64_t i = (int64_t)(g.b + (g.r0 + r) / a.p.G) * a.p.Hq + g.h0 + (g.r0 + r) % a.p.G;
        if (whole) {
            store4(q.whole + i * D + c, y);
            if (c == 0) q.ml[i] = make_float2(M, L);
        } else {
            store4(rec + r * D + c, y);
            if (c == 0) {
                rec[kRows * D + r] = M;
                rec[kRows * D + kRows + r] = L;
            }
        }
        if (c == 0 && (whole || g.k == 0)) q.desc[i] = whole ? make_int4(1, 0, 0, 0) : make_int4(g.np, 2 * g.c0 + g.s0, r, 1);
    } else if (whole) {
        // (no token seen: o = 0; scores that are all minus infinity: 0 / 0)
        const float inv = L == 0.f ? (sees_any(a, g.b) ? NAN : 0.f) : 1.f / L;
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] *= inv;
        store4(reinterpret_cast<T*>(a.O.data) + (int64_t)g.b * a.O.row + (int64_t)(g.h0 + r) * a.O.head + c, y);
        if (a.lse && c == 0) a.lse[(int64_t)g.b * a.p.Hq + g.h0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kAttnLn2;
    } else {
        store4(rec + r * D + c, y);
        if (c == 0) {
            rec[kRows * D + r] = M;
            rec[kRows * D + kRows + r] = L;
        }
    }
}

// ---- the join of an item's pieces ----
// Up to 16 pieces are joined at once, by the last of them to arrive; an item of more pieces takes a
// second round over those joins.  A join counts its arrivals in a cell that holds the call's tag (56
// bits) and the count (8): whoever takes part first swaps whatever the workspace held for the tag and a
// count of 0 -- long before its own arrival, off the critical path -- and the last one leaves 0.  So a
// workspace needs no clearing, and a replayed graph, whose tag stays the same, finds no old count: every
// piece is counted, those of a CTA whose waits gave up too (settle).
template <int D>
__device__ __forceinline__ void open_cell(const Args& a, int piece, int slot) {
    unsigned long long* c = cell<D>(a, piece, slot);
    const unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(c);
    if ((old ^ a.tag) >> 8) atomicCAS(c, old, (unsigned long long)a.tag);   // (a failure: another one was faster)
}
template <int D>
__device__ __forceinline__ void open_cells(const Args& a, const Seg& g) {
    const int first = g.k / kJoin * kJoin;
    open_cell<D>(a, g.c0 + first, first == 0 ? g.s0 : 0);
    if (g.np > kJoin) open_cell<D>(a, g.c0, 2 + g.s0);
}

// A join that piece k of an item takes part in: pieces c0 + step (first + x), x < cnt, the very first one's record
// in slot0.
struct Join {
    int k, np, step, slot0, slot;
    __device__ __forceinline__ explicit Join(const Seg& g) : k(g.k), np(g.np), step(1), slot0(g.s0), slot(0) {}
    __device__ __forceinline__ int first() const { return k / kJoin * kJoin; }
    __device__ __forceinline__ int cnt() const { return min(kJoin, np - first()); }
    __device__ __forceinline__ int head(const Seg& g) const { return g.c0 + step * first(); }
    __device__ __forceinline__ int hslot() const { return first() == 0 ? slot0 : slot; }
    // the second round: the joins, each in a record of its first piece
    __device__ __forceinline__ void next() {
        k /= kJoin;
        np = (np + kJoin - 1) / kJoin;
        step = kJoin;
        slot0 = 2 + slot0;
        slot = 2;
    }
};
// One more arrival; whether it is the last one of `cnt`.
template <int D>
__device__ __forceinline__ bool arrive(const Args& a, int head, int hslot, int cnt) {
    unsigned long long* c = cell<D>(a, head, hslot);
    unsigned long long old;
    asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(reinterpret_cast<uint64_t>(c)) : "memory");
    const bool last = (int)(old & 255) == cnt - 1;
    if (last) *reinterpret_cast<volatile unsigned long long*>(c) = 0ull;
    return last;
}

// Segment g's record is written by this group's NT threads (numbered t).  `bar` is their barrier.
template <typename T, int D, int NT, typename F>
__device__ void join_pieces(const Args& a, const Seg& g, int t, int* go, int* arrived, F&& bar) {
    for (Join join(g);; join.next()) {
        const int first = join.first(), cnt = join.cnt(), head = join.head(g), hslot = join.hslot(), slot = join.slot;
        const int np = join.np, step = join.step;
        bar();
        if (t == 0) {
            *go = arrive<D>(a, head, hslot, cnt);
            if (step == 1) arrived[g.k == 0 ? g.s0 : 0] = 1;
        }
        bar();
        if (!*go) return;
        const float* rec0 = record<D>(a, head, hslot);
        const int64_t stride = (int64_t)step * kSlots * record_floats(D);    // from a member's record to the next
        const int64_t shift = (int64_t)(slot - hslot) * record_floats(D);    // (the first may sit in another slot)
        for (int e = t; e < g.R * (D / 4); e += NT) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            float m[kJoin], l[kJoin];
            float4 z[kJoin];
#pragma unroll
            for (int x = 0; x < kJoin; ++x) {
                const float* rec = rec0 + x * stride + (x > 0 ? shift : 0);
                m[x] = x < cnt ? __ldcg(rec + kRows * D + r) : -INFINITY;
                l[x] = x < cnt ? __ldcg(rec + kRows * D + kRows + r) : 0.f;
                z[x] = x < cnt ? __ldcg(reinterpret_cast<const float4*>(rec + r * D + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float M = -INFINITY, L = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < kJoin; ++x) M = fmaxf(M, m[x]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int x = 0; x < kJoin; ++x) {
                const float f = ex2(m[x] - base);
                L = fmaf(f, l[x], L);
                y[0] = fmaf(f, z[x].x, y[0]);
                y[1] = fmaf(f, z[x].y, y[1]);
                y[2] = fmaf(f, z[x].z, y[2]);
                y[3] = fmaf(f, z[x].w, y[3]);
            }
            write_out<T, D, false>(a, g, cnt == np, record<D>(a, head, 2 + hslot), r, c, y, M, L);
        }
        if (cnt == np) return;
    }
}

// The end of a CTA whose waits gave up (all threads, after all roles): no copy is left in flight, and its pieces
// that were not counted are, so that every cell of the call ends at 0 (what the joins then make of their records
// is as invalid as the call).
template <int D, int S, int NS, bool SH, int NT = kThreads, int TILE = kTile, bool PRE = false, typename B>
__device__ __noinline__ void settle(const Args& a, B& bars) {
    if (threadIdx.x == 0) {
        const int n = max(bars.issued, bars.ahead), i = bars.given;
        // (of a tile's copies, those of a warp that met the end sooner are missing, or the tile is not armed: then the others are
        // waited for for long enough)
        for (int x = max(0, n - S); x < n; ++x) mbar_wait(smem_u32(&bars.full[x % S]), (uint32_t)(x / S) & 1, kDrainNs);
        for (int x = max(0, i - NS); x < i; ++x) mbar_wait(smem_u32(&bars.seg_full[x % NS]), (uint32_t)(x / NS) & 1, kWaitNs);
    }
    if constexpr (SH) return;                                      // (nothing is counted)
    Start st;
    if (!find_start<false, NT, TILE, kRows, PRE>(a, &st) || threadIdx.x != 0) return;
    int ignored = 0;
    auto count = [&](int b) { return item_tiles<TILE, PRE>(a, b, paged_tokens(a.p, a.p.kv_len[b]), &ignored); };
    int b = st.b, tiles = count(b);
    int item = (int)(st.rem / tiles), t0 = (int)(st.rem % tiles);
    for (int64_t u = st.u0; u < st.u1;) {
        const int t1 = (int)min((int64_t)tiles, t0 + (st.u1 - u));
        if (t0 > 0 || t1 < tiles) {
            Seg g;
            place_piece(st, u - t0, tiles, &g);
            if (!bars.arrived[g.k == 0 ? g.s0 : 0]) {
                open_cells<D>(a, g);
                for (Join join(g); arrive<D>(a, join.head(g), join.hslot(), join.cnt()) && join.cnt() < join.np;) join.next();
            }
        }
        u += t1 - t0;
        t0 = 0;
        if (++item == a.I && u < st.u1) {
            item = 0;
            tiles = count(++b);
        }
    }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

inline Args make_args(const DecodeArgs& d) {
    Args a;
    a.p = d.p;
    a.pre = d.pre;
    a.sh = d.sh;
    a.parts = d.parts;
    a.Q = d.Q;
    a.O = d.O;
    a.lse = d.lse;
    a.part = d.part;
    a.tag = d.tag << 8;
    a.scale_log2 = d.scale_log2;
    a.give_up = d.give_up;
    a.RG = (d.p.G + kRows - 1) / kRows;
    a.I = d.p.Hkv * a.RG;
    return a;
}

template <typename T, int D, typename K>
cudaError_t launch_kernel(K kernel, int warps, std::atomic<uint64_t>& done, const DecodeArgs& d, cudaStream_t st,
                          int smem = Cfg<T, D>::kSmem) {
    using C = Cfg<T, D>;
    Maps maps;
    const auto ty = sizeof(T) == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                    : sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int64_t depth = (int64_t)d.p.n_pages * d.p.Hkv;
    const int rows = d.p.page < C::kTokens ? d.p.page : C::kTokens;
    // (e4m3: rows of 128 bytes)
    const int wide = sizeof(T) == 1 ? 128 : D, fold = wide / D;
    if (!make_tmap_pages(&maps.k, ty, sizeof(T), d.p.K, wide, d.p.page / fold, depth, rows / fold, wide * (int)sizeof(T) / 128) ||
        !make_tmap_pages(&maps.v, ty, sizeof(T), d.p.V, wide, d.p.page / fold, depth, rows / fold, wide * (int)sizeof(T) / 128))
        return cudaErrorInvalidValue;
    cudaError_t e = opt_in_smem(kernel, smem, done);
    if (e != cudaSuccess) return e;
    return launch_behind(kernel, kPieces, warps * kWarp, smem, st, maps, make_args(d));
}

}  // namespace
}  // namespace lola
